// linear.hip -- feature projections y = act(x W^T + bias) + residual and
// their gradients around the tiled product (linear_tile.h): few rows without
// tiles, dz = dy act'(z) with the bias gradient, copies of rows that do not
// start at 16-byte boundaries, and the sum of partial products.
#include "elem.h"

#include <type_traits>

namespace haste {

namespace {

constexpr int NT = 256;
inline size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == 0) return 1.f;
    if (ACT == 1) return z > 0.f ? 1.f : z != z ? z : 0.f;
    // s + z s (1 - s) t', s = sigmoid(t); 1 - s from its own exponential's side
    constexpr float c = 2.0f * 0.7978845608028654f;
    const float t = ACT == 3 ? z : z * __builtin_fmaf(z * z, c * 0.044715f, c);
    const float dt = ACT == 3 ? 1.f : __builtin_fmaf(z * z, 3.f * c * 0.044715f, c);
    const float e = __builtin_amdgcn_exp2f(-fabsf(t) * kLog2e), r = __builtin_amdgcn_rcpf(1.f + e);
    const float s = t >= 0.f ? r : e * r, o = t >= 0.f ? e * r : r;
    // far out s (1 - s) is 0 where z and t' may be infinite
    const float d = s * o;
    return d > 0.f ? __builtin_fmaf(z * d, dt, s) : z != z ? z : s;
}

__device__ __forceinline__ float activate_any(int act, float z) {
    if (act == 0) return z;
    if (act == 1) return z > 0.f ? z : z != z ? z : 0.f;
    constexpr float c = 2.0f * 0.7978845608028654f * kLog2e;
    const float t = act == 3 ? z * -kLog2e : z * __builtin_fmaf(z * z, -c * 0.044715f, -c);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

// 16 bytes of a row from element k; past its end (K) zeros
template <bool BF>
__device__ __forceinline__ u32x4 piece(const void *row, int k, int K) {
    constexpr int P = BF ? 8 : 4;
    if (k + P <= K) return BF ? (u32x4) * (const u32x4h *)((const unsigned short *)row + k) : (u32x4) * (const u32x4w *)((const unsigned *)row + k);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < P - 1; ++j)
        if (k + j < K) {
            if (BF) v[j >> 1] |= (unsigned)((const unsigned short *)row)[k + j] << (16 * (j & 1));
            else v[j] = ((const unsigned *)row)[k + j];
        }
    return v;
}

}  // namespace

// --------------------------------------------------------------- few rows
// Up to 16 NB rows of x: the weights' bytes count.  A workgroup takes 16
// columns n, its four waves a quarter of k each in turns, streaming the
// weights' rows straight into MFMA operands; the waves' sums meet in LDS.  fp32
// operands: a wave's runs of 128 k are summed by themselves, as the tiles' runs
// are (K = 4096: 2.2e-7 from the exact sums, one chain of K / 4 5.9e-7).
// 1 x 1024 -> 1024 bf16: 5.3 us, of which 2.5 are the launch; 4096 -> 4096 16 us a
// call, 2.1 TB/s.
template <bool BF, bool YB, int NB>
__global__ __launch_bounds__(256) void k_linear_few(LinearArgs a) {
    constexpr int P = BF ? 8 : 4, STEP = 4 * P, U = 8;     // elements of a piece, of a step
    __shared__ float part[4][NB][64][5];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    constexpr size_t E = BF ? 2 : 4;
    const int n0 = blockIdx.x * 16;
    const char *pw = (const char *)a.W + (size_t)min(n0 + r, a.N - 1) * a.K * E;
    const char *px[NB];
    f32x4 acc[NB], total[NB];                              // total: of fp32 runs
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        total[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
        px[b] = (const char *)a.x + (size_t)min(16 * b + r, a.M - 1) * a.ldx * E;
        acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    auto step = [&](u32x4 fw, u32x4 fx, int b) {
        if (BF) {
            acc[b] = mfma32(__builtin_bit_cast(bf16x8, fw), __builtin_bit_cast(bf16x8, fx), acc[b]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fw[j]), __uint_as_float(fx[j]), acc[b], 0, 0, 0);
        }
    };
    for (int k0 = w * STEP; k0 < a.K; k0 += 4 * U * STEP) {
        u32x4 fw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) fw[i] = piece<BF>(pw, k0 + 4 * i * STEP + P * q, a.K);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (k0 + 4 * i * STEP >= a.K) break;
#pragma unroll
            for (int b = 0; b < NB; ++b) step(fw[i], piece<BF>(px[b], k0 + 4 * i * STEP + P * q, a.K), b);
        }
        if (!BF) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                total[b] += acc[b];
                acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[w][b][lane][e] = (BF ? acc : total)[b][e];
    __syncthreads();
    if (w >= NB) return;
    const int m = 16 * w + r;      // the wave's row tile
    if (m >= a.M) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = n0 + 4 * q + e;
        if (n >= a.N) break;
        float v = (part[0][w][lane][e] + part[1][w][lane][e]) + (part[2][w][lane][e] + part[3][w][lane][e]);
        if (a.bias) v += a.bbf ? load1<true>(a.bias, n) : load1<false>(a.bias, n);
        const int64_t o = (int64_t)m * a.N + n;
        if (a.zout) store1<YB>(a.zout, o, v);
        v = activate_any(a.act, v);
        if (a.res) v += load1<YB>(a.res, o);
        store1<YB>(a.y, o, v);
    }
}

// ------------------------------------------------- dz and the bias gradient
// dz = dy act'(z) in x's type, rows of Np (zeros past N), and the columns' sums
// of the unrounded values over the workgroup's rows.  A wave a row, a lane
// eight columns; blockIdx.y takes the columns past 512.  Bound by memory: 65536 x
// 1024 bf16 78 to 84 us, 4.8 to 5.1 TB/s.  Narrow rows leave lanes idle and are
// bound by its latency: the bias gradient of 65536 x 16 to 512 takes 50 to 56 us.
// dz in x's type: bf16 products take bf16 operands, and the layer's own dZ is
// rounded so.  Of a bf16 dy this is as many bits as it came with; dx and dW are 1.2
// and 1.4 times as far from the exact ones as from an unrounded dz (1.9e-3 and
// 2.3e-3 against 1.7e-3, a bf16 result's own rounding).  fp32 operands keep all of it.
struct DzArgs {
    const void *dy, *z;
    void *dz;                // or null
    float *part;             // gridDim.x x N, or null
    int M, N, Np;
};
template <bool XB, bool YB, int ACT>
__global__ __launch_bounds__(NT) void k_linear_dz(DzArgs a) {
    __shared__ float s[4][64][9];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = 8 * (64 * (int)blockIdx.y + lane);
    const bool tail = a.N & 7;
    float sum[8] = {};
    constexpr int U = 2;
    for (int64_t r0 = (int64_t)blockIdx.x * 4 + w; r0 < a.M; r0 += (int64_t)gridDim.x * 4 * U) {
        Raw8<YB> g[U], z[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t r = r0 + (int64_t)i * gridDim.x * 4;
            g[i] = raw8n<YB>(a.dy, r * a.N + c, c, r < a.M ? a.N : 0, tail);
            if (ACT) z[i] = raw8n<YB>(a.z, r * a.N + c, c, r < a.M ? a.N : 0, tail);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t r = r0 + (int64_t)i * gridDim.x * 4;
            const int N = r < a.M ? a.N : 0;
            float v[8], t[8];
            unpack8n<YB>(g[i], c, N, tail, v);
            if (ACT) {
                unpack8n<YB>(z[i], c, N, tail, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = j < N - c ? v[j] * act_slope<ACT>(t[j]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += v[j];
            if (a.dz && r < a.M && c < a.Np) store8<XB>(a.dz, r * a.Np + c, v);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[w][lane][j] = sum[j];
    __syncthreads();
    if (w == 0 && c < a.N) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = (s[0][lane][j] + s[1][lane][j]) + (s[2][lane][j] + s[3][lane][j]);
        store8n<false>(a.part, (int64_t)blockIdx.x * a.N + c, a.N - c, sum);
    }
}

// The columns' partial sums added up: 16 waves of 64 columns, a sixteenth of
// the partials each, joined in LDS.
__global__ __launch_bounds__(1024) void k_linear_bias_sum(const float *part, int parts, int N, float *db, bool accumulate) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float t = 0.f;
    if (c < N) {
        constexpr int U = 8;
        for (int p0 = w; p0 < parts; p0 += 16 * U) {
            float v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = p0 + 16 * i < parts ? part[(int64_t)(p0 + 16 * i) * N + c] : 0.f;
#pragma unroll
            for (int i = 0; i < U; ++i) t += v[i];
        }
    }
    s[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < N) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += s[i][lane];
        db[c] = accumulate ? db[c] + t : t;
    }
}

// ------------------------------------------------------------ small passes
// rows of C elements to rows of Cp (a multiple of eight), zeros past the end
template <bool BF>
__global__ __launch_bounds__(NT) void k_linear_pad(const void *x, int64_t ld, int64_t rows, int C, int Cp, void *to) {
    const unsigned nv = (unsigned)Cp / 8;
    const bool tail = C & 7;
    for (uint64_t i = (uint64_t)blockIdx.x * NT + threadIdx.x; i < (uint64_t)rows * nv; i += (uint64_t)gridDim.x * NT) {
        const int64_t r = (int64_t)(i / nv);
        const int c = 8 * (int)(i % nv);
        float v[8];
        unpack8n<BF>(raw8n<BF>(x, r * ld + c, c, C, tail), c, C, tail, v);
        store8<BF>(to, r * Cp + c, v);
    }
}

// the sum of `splits` partial products, in their order; added to what is there
template <bool BF>
__global__ __launch_bounds__(NT) void k_linear_sum(const float *part, int splits, int64_t n, void *to, bool accumulate) {
    const int64_t i = 4 * ((int64_t)blockIdx.x * NT + threadIdx.x);
    if (i >= n) return;
    const int m = (int)min((int64_t)4, n - i);
    float s[4] = {};
    constexpr int U = 8;
    for (int p0 = 0; p0 < splits; p0 += U) {
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if (p0 + u < splits) {
                const float *p = part + (p0 + u) * n + i;
                if (m == 4) v[u] = *(const f32x4u *)p;
                else
                    for (int e = 0; e < m; ++e) v[u][e] = p[e];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += v[u][e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < m) store1<BF>(to, i + e, accumulate ? load1<BF>(to, i + e) + s[e] : s[e]);
}

namespace {

// Rows that take no tiles, us a call against 64 x 64 tiles.  1024 -> 1024 bf16: 16
// rows 7.1 and 8.2, 32 6.9 and 7.9, 48 8.2 and 7.9, fp32 32 rows 10.1 and 25; 4096 ->
// 4096 bf16: 16 rows 16.1 and 34.5, 32 27.4 and 34.4, 48 42 and 33.8, fp32 32 rows 55
// and 90.
constexpr int kFewRows = 32;

bool on16(const void *p, int64_t ld, bool bf) { return (uintptr_t)p % 16 == 0 && ld % (bf ? 8 : 4) == 0; }
inline int round8(int n) { return (n + 7) & ~7; }
inline size_t es(bool bf) { return bf ? 2 : 4; }

// rows that the tiles read where they lie: 16-byte boundaries, whole pieces
bool direct(const void *p, int64_t ld, int cols, bool bf) { return on16(p, ld, bf) && cols % (bf ? 8 : 4) == 0; }

// Runs of the contraction of a weight gradient of N x K, each to a partial product
// of its own.  bf16: as many as give every CU a tile of 256 x 256 where they are
// of 2048 rows and more (65536 x 1024 x 768: 21 runs 113 us, 8 with tiles of 128
// x 128 132; 16384 rows of it: 16 runs 48, 6 to 8 with the smaller tiles 42);
// otherwise as many as give every CU a tile of 128 x 128, of 1024 rows and more
// (8192 x 1024 x 1024: 1, 2, 4, 8 runs 41, 40, 30, 33; 2048 x 512 x 768: 13.5, 14,
// 14.4, 18).  fp32: none where 128 x 128 tiles fill the CUs, otherwise tiles of
// 64 x 64, eight a CU, and runs of 512 rows and more (4001 x 513 x 1001: 7 runs
// 68, 12 with the larger tiles 83; 16384 x 768 x 768: 13 runs 177, 12 with the
// larger tiles 195; 512 x 768 x 768: 1 run 14, 2 and 3 runs 20).  Runs are whole
// multiples of 128 rows.
void dw_splits(bool bf, int M, int N, int K, int *splits, int *run) {
    auto tiles = [&](int64_t t) { return (((int64_t)N + t - 1) / t) * (((int64_t)K + t - 1) / t); };
    const int64_t big = tiles(256), mid = tiles(128);
    int64_t s;
    if (bf) {
        s = big < 256 ? 256 / big : 1;
        if (M / s < 2048 || big * s < 192) s = min((256 + mid - 1) / mid, (int64_t)M / 1024);
    } else {
        s = mid >= 192 ? 1 : min(2048 / tiles(64), (int64_t)M / 512);
    }
    if (s < 1) s = 1;
    int64_t r = ((int64_t)M + s - 1) / s;
    r = (r + 127) / 128 * 128;
    if (r > (1 << 24)) r = 1 << 24;
    *run = (int)r;
    *splits = (int)((M + r - 1) / r);
}
constexpr int kBiasParts = 256;
int bias_parts(int M) { return M < 4 * kBiasParts ? (M + 3) / 4 : kBiasParts; }

struct BwdPlan {
    bool pad_x, pad_w, own_dz;
    int Np, splits, run;
    size_t dz, x, w, part, bias, total;
};
BwdPlan bwd_plan(const LinearArgs &a) {
    BwdPlan p{};
    const size_t e = es(a.xbf);
    p.pad_x = a.dW && !direct(a.x, a.ldx, a.K, a.xbf);
    p.pad_w = a.dx && !direct(a.W, a.K, a.K, a.xbf);
    p.own_dz = (a.dx || a.dW) && (a.act != 0 || a.xbf != a.ybf || !direct(a.dy, a.N, a.N, a.ybf));
    p.Np = p.own_dz ? round8(a.N) : a.N;
    dw_splits(a.xbf, a.M, a.N, a.K, &p.splits, &p.run);
    size_t o = 0;
    p.dz = o;
    if (p.own_dz) o += up((size_t)a.M * p.Np * e);
    p.x = o;
    if (p.pad_x) o += up((size_t)a.M * round8(a.K) * e);
    p.w = o;
    if (p.pad_w) o += up((size_t)a.N * round8(a.K) * e);
    p.part = o;
    if (a.dW && p.splits > 1) o += up((size_t)p.splits * a.N * a.K * 4);
    p.bias = o;
    if (a.db) o += up((size_t)bias_parts(a.M) * a.N * 4);
    p.total = o;
    return p;
}

void pad(bool bf, const void *x, int64_t ld, int64_t rows, int C, void *to, hipStream_t st) {
    const int64_t want = (rows * (round8(C) / 8) + NT - 1) / NT;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536));
    if (bf) hipLaunchKernelGGL(k_linear_pad<true>, grid, dim3(NT), 0, st, x, ld, rows, C, round8(C), to);
    else hipLaunchKernelGGL(k_linear_pad<false>, grid, dim3(NT), 0, st, x, ld, rows, C, round8(C), to);
}

template <bool XB, bool YB>
void dz_pass(int act, const DzArgs &d, dim3 grid, hipStream_t st) {
#define GO(A) hipLaunchKernelGGL((k_linear_dz<XB, YB, A>), grid, dim3(NT), 0, st, d)
    if (act == 0) GO(0);
    else if (act == 1) GO(1);
    else if (act == 2) GO(2);
    else GO(3);
#undef GO
}

}  // namespace

size_t linear_fwd_ws_bytes(const LinearArgs &a) {
    if (a.M <= kFewRows) return 0;
    const size_t e = es(a.xbf), kp = (size_t)round8(a.K) * e;
    return (direct(a.x, a.ldx, a.K, a.xbf) ? 0 : up(a.M * kp)) + (direct(a.W, a.K, a.K, a.xbf) ? 0 : up(a.N * kp));
}

hipError_t launch_linear_fwd(const LinearArgs &a, hipStream_t st) {
    if (a.M <= kFewRows) {
        const dim3 grid((unsigned)((a.N + 15) / 16));
        auto go = [&](auto nb) {
            constexpr int NB = decltype(nb)::value;
            if (a.xbf && a.ybf) hipLaunchKernelGGL((k_linear_few<true, true, NB>), grid, dim3(256), 0, st, a);
            else if (a.xbf) hipLaunchKernelGGL((k_linear_few<true, false, NB>), grid, dim3(256), 0, st, a);
            else hipLaunchKernelGGL((k_linear_few<false, false, NB>), grid, dim3(256), 0, st, a);
        };
        if (a.M <= 16) go(std::integral_constant<int, 1>{});
        else go(std::integral_constant<int, 2>{});
        return hipGetLastError();
    }
    LinArgs g{};
    char *ws = (char *)a.ws;
    const int kp = round8(a.K);
    g.P = a.x;
    g.ldp = a.ldx;
    g.Q = a.W;
    g.ldq = a.K;
    if (!direct(a.x, a.ldx, a.K, a.xbf)) {
        pad(a.xbf, a.x, a.ldx, a.M, a.K, ws, st);
        g.P = ws;
        g.ldp = kp;
        ws += up((size_t)a.M * kp * es(a.xbf));
    }
    if (!direct(a.W, a.K, a.K, a.xbf)) {
        pad(a.xbf, a.W, a.K, a.N, a.K, ws, st);
        g.Q = ws;
        g.ldq = kp;
    }
    g.M = a.M;
    g.N = a.N;
    g.K = a.K;
    g.splits = 1;
    g.k_split = a.K;
    g.C = a.y;
    g.ldc = a.N;
    g.bias = a.bias;
    g.bias_bf = a.bbf;
    g.res = a.res;
    g.ldr = a.N;
    g.Z = a.zout;
    return a.xbf ? launch_linear_bf16(g, true, true, a.ybf, a.act, st) : launch_linear_f32(g, true, true, a.act, st);
}

size_t linear_bwd_ws_bytes(const LinearArgs &a) { return bwd_plan(a).total; }

hipError_t launch_linear_bwd(const LinearArgs &a, hipStream_t st) {
    const BwdPlan p = bwd_plan(a);
    char *ws = (char *)a.ws;
    const void *dz = a.dy;
    if (p.own_dz || a.db) {
        DzArgs d{a.dy, a.z, p.own_dz ? ws + p.dz : nullptr, a.db ? (float *)(ws + p.bias) : nullptr, a.M, a.N, p.Np};
        const dim3 grid(bias_parts(a.M), (unsigned)((a.N + 511) / 512));
        if (a.xbf && a.ybf) dz_pass<true, true>(a.act, d, grid, st);
        else if (a.xbf) dz_pass<true, false>(a.act, d, grid, st);
        else dz_pass<false, false>(a.act, d, grid, st);
        if (a.db)
            hipLaunchKernelGGL(k_linear_bias_sum, dim3((unsigned)((a.N + 63) / 64)), dim3(1024), 0, st, (const float *)d.part,
                               (int)grid.x, a.N, a.db, a.accumulate);
        if (p.own_dz) dz = d.dz;
    }
    const int kp = round8(a.K);
    LinArgs g{};
    g.P = dz;
    g.ldp = p.Np;
    g.splits = 1;
    if (a.dx) {
        g.Q = a.W;
        g.ldq = a.K;
        if (p.pad_w) {
            pad(a.xbf, a.W, a.K, a.N, a.K, ws + p.w, st);
            g.Q = ws + p.w;
            g.ldq = kp;
        }
        g.M = a.M;
        g.N = a.K;
        g.K = g.k_split = a.N;
        g.C = a.dx;
        g.ldc = a.lddx;
        g.res = a.add;
        g.ldr = a.K;
        const hipError_t e = a.xbf ? launch_linear_bf16(g, true, false, true, 0, st) : launch_linear_f32(g, true, false, 0, st);
        if (e != hipSuccess) return e;
    }
    if (a.dW) {
        g.Q = a.x;
        g.ldq = a.ldx;
        if (p.pad_x) {
            pad(a.xbf, a.x, a.ldx, a.M, a.K, ws + p.x, st);
            g.Q = ws + p.x;
            g.ldq = kp;
        }
        g.M = a.N;
        g.N = a.K;
        g.K = a.M;
        g.splits = p.splits;
        g.k_split = p.run;
        const bool parts = p.splits > 1;
        g.C = parts ? ws + p.part : a.dW;
        g.ldc = a.K;
        g.res = a.accumulate && !parts ? a.dW : nullptr;
        g.ldr = a.K;
        const hipError_t e = a.xbf ? launch_linear_bf16(g, false, false, !parts, 0, st) : launch_linear_f32(g, false, false, 0, st);
        if (e != hipSuccess) return e;
        if (parts) {
            const int64_t n = (int64_t)a.N * a.K;
            const dim3 grid((unsigned)((n / 4 + NT) / NT));
            if (a.xbf) hipLaunchKernelGGL(k_linear_sum<true>, grid, dim3(NT), 0, st, (const float *)g.C, p.splits, n, a.dW, a.accumulate);
            else hipLaunchKernelGGL(k_linear_sum<false>, grid, dim3(NT), 0, st, (const float *)g.C, p.splits, n, a.dW, a.accumulate);
        }
    }
    return hipGetLastError();
}

}  // namespace haste
