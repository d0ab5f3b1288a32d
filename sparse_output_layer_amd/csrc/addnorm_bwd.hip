// addnorm_bwd.hip -- gradients of a block's output joined to the residual
// stream between two layer norms (addnorm.hip), in one pass over the rows:
//
//   h2 = (r' - m2) s2, u = dy g2, dR = dr' + s2 (u - mean(u) - h2 mean(u h2))
//   dr = dR, a = drop(alpha gate dR), dgate = alpha dR drop(p)
//   h1 = (o - m1) s1, v = a g1, do = post ? s1 (v - mean(v) - h1 mean(v h1)) : a
//   dg2 = sum dy h2, db2 = sum dy, dg1 = sum a h1, db1 = sum a   (over the rows)
//
// Bound by memory: r', dy, dr', o in, dr and do out, a row staying in the
// registers of the threads that share it: 40001 x 1001, a gate for every row, 183
// us, 4.9 TB/s; 512 x 768 9.2 and 5.2.  The weight gradients are summed over
// a workgroup's rows in registers, its threads' sums joined in LDS, and the
// workgroups' partial sums added up by a second launch, all in a fixed order.
// Four sums of D serve all five: with t = alpha drop(dR) and a gate of all rows,
//   db1 = gate sum t, dg1 = gate sum t h1, dgate = g1 sum t h1 + b1 sum t
// (h1 = o, g1 = 1, b1 = 0 without the post norm); with a gate for every row
// the sums run over a instead of t.
#include "rows.h"

namespace haste {

namespace {

constexpr int NT = 256;
constexpr int NB = 256;       // threads of a workgroup whose rows are shorter
enum { DYH, DY, TH, T, KINDS };     // sum dy h2, sum dy, sum t h1, sum t

// which partial sums a call has
__host__ __device__ __forceinline__ bool has(const AddNormArgs &a, int kind) {
    const bool gate = a.dgate && !a.gate_rows;
    return kind == DYH ? a.dg2 != nullptr : kind == DY ? a.db2 != nullptr
         : kind == TH ? a.dg1 || gate : a.db1 || (gate && a.post);
}
__host__ __device__ __forceinline__ bool columns_of(const AddNormArgs &a) {
    return has(a, DYH) || has(a, DY) || has(a, TH) || has(a, T);
}

// what dropout multiplies the eight elements of vector v of row r by
__device__ __forceinline__ void keep8(const DropArgs &d, unsigned v, unsigned r, float *k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = 1.f;
    if (d.thr) drop8(d, v, r, k);
}
// a dropped element is 0 whatever it was
__device__ __forceinline__ float kept(float k, float x) { return k != 0.f ? k * x : 0.f; }

}  // namespace

template <bool OB, bool RB, bool YB, bool TAIL, int NV, int TPR>
__global__ __launch_bounds__(TPR > NB ? TPR : NB) void k_addnorm_bwd(AddNormArgs a) {
    constexpr int NTH = TPR > NB ? TPR : NB, RW = NTH / TPR;
    __shared__ float s[2][NTH / 64], q[2][NTH / 64];
    __shared__ __attribute__((aligned(16))) float acc[RW][8 * NV * TPR];
    // the weights of short rows lie in LDS, those of others are read from L2 for
    // every row: in registers they would leave no room for the row and the sums
    constexpr bool LDS = TPR <= 256;
    constexpr int COLS = 8 * NV * TPR;
    __shared__ __attribute__((aligned(16))) float sw[LDS ? 4 * COLS : 4];
    int turn = 0;
    const int li = threadIdx.x % TPR, tail = tail_of<TAIL, TPR>(a.D);
    const bool columns = columns_of(a);
    auto weight = [&](int i, int c, float *w) {
        const void *p = i == 0 ? a.g2 : i == 1 ? (a.gate_rows ? nullptr : a.gate) : a.post ? (i == 2 ? a.g1 : a.b1) : nullptr;
        load_w8(p, a.wbf, c, a.D, i == 3 ? 0.f : 1.f, w);
    };
    if (LDS) {
        for (int c = 8 * threadIdx.x; c < COLS; c += 8 * NTH)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w[8];
                weight(i, c, w);
#pragma unroll
                for (int e = 0; e < 8; e += 4) *(f32x4 *)(sw + i * COLS + c + e) = (f32x4){w[e], w[e + 1], w[e + 2], w[e + 3]};
            }
        __syncthreads();
    }
    // gamma, gate, gamma_post, beta_post (i = 0 .. 3) of the eight columns from c
    auto get = [&](int i, int c, float *w) {
        if (!LDS) {
            weight(i, c, w);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const f32x4 x = *(const f32x4 *)(sw + i * COLS + c + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[e + j] = x[j];
        }
    };
    float sum[KINDS][NV][8];
#pragma unroll
    for (int i = 0; i < KINDS; ++i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[i][k][j] = 0.f;
    const float inv = 1.f / (float)a.D;
    for (int64_t rb = (int64_t)blockIdx.x * RW; rb < a.B; rb += (int64_t)gridDim.x * RW) {
        const int64_t r = rb + threadIdx.x / TPR;
        const bool live = r < a.B;
        const int D = live ? a.D : 0, lw = opaque_index(li);
        Raw8<RB> xr[NV], gr[NV];
        Raw8<YB> yr[NV];
        Raw8<OB> orw[NV], gt[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (li + k * TPR);
            const bool t = TAIL && k == tail;
            const int64_t i = r * a.D + c;
            if (a.norm) {
                xr[k] = raw8n<RB>(a.r_out, i, c, D, t);
                yr[k] = raw8n<YB>(a.dy, i, c, D, t);
            }
            if (a.dr_out) gr[k] = raw8n<RB>(a.dr_out, i, c, D, t);
            orw[k] = raw8n<OB>(a.o, i, c, D, t);
            if (a.gate_rows) gt[k] = raw8n<OB>(a.gate, i, c, D, t);
        }
        float dR[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (a.dr_out) {
                unpack8n<RB>(gr[k], 8 * (li + k * TPR), a.D, TAIL && k == tail, dR[k]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) dR[k][j] = 0.f;
            }
        }
        if (a.norm) {
            const float mean = live ? a.stats[2 * (int64_t)a.B + r] : 0.f, rstd = live ? a.stats[3 * (int64_t)a.B + r] : 0.f;
            float h[NV][8], g[NV][8], sg = 0.f, sgh = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = 8 * (li + k * TPR), n = D - c;
                float w[8];
                unpack8n<RB>(xr[k], c, a.D, TAIL && k == tail, h[k]);
                unpack8n<YB>(yr[k], c, a.D, TAIL && k == tail, g[k]);
                get(0, 8 * (lw + k * TPR), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[k][j] = (TAIL ? j < n : n > 0) ? (h[k][j] - mean) * rstd : 0.f;
                    sum[DYH][k][j] = __builtin_fmaf(g[k][j], h[k][j], sum[DYH][k][j]);
                    sum[DY][k][j] += g[k][j];
                    g[k][j] *= w[j];
                    sg += g[k][j];
                    sgh = __builtin_fmaf(g[k][j], h[k][j], sgh);
                }
            }
            row_sum2<TPR, NTH>(sg, sgh, s, q, turn);
            sg *= inv;
            sgh *= inv;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) dR[k][j] += rstd * (g[k][j] - sg - h[k][j] * sgh);
        }
        const float m1 = live && a.post ? a.stats[r] : 0.f, s1 = a.post ? (live ? a.stats[a.B + r] : 0.f) : 1.f;
        float h[NV][8], g[NV][8], sg = 0.f, sgh = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = li + k * TPR, c = 8 * v, n = D - c;
            float w[8], keep[8], gate[8], b1[8];
            unpack8n<OB>(orw[k], c, a.D, TAIL && k == tail, h[k]);
            if (a.gate_rows) unpack8n<OB>(gt[k], c, a.D, TAIL && k == tail, gate);
            else get(1, 8 * (lw + k * TPR), gate);
            get(2, 8 * (lw + k * TPR), w);
            get(3, 8 * (lw + k * TPR), b1);
            keep8(a.drop, (unsigned)v, (unsigned)r, keep);
            float dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = TAIL ? j < n : n > 0;
                h[k][j] = in ? (h[k][j] - m1) * s1 : 0.f;
                const float t = in ? kept(keep[j], a.alpha * dR[k][j]) : 0.f;
                const float e = in && keep[j] != 0.f ? gate[j] * t : 0.f;
                const float x = a.gate_rows ? e : t;
                dg[j] = in && keep[j] != 0.f ? t * __builtin_fmaf(h[k][j], w[j], b1[j]) : 0.f;
                sum[TH][k][j] = keep[j] != 0.f ? __builtin_fmaf(x, h[k][j], sum[TH][k][j]) : sum[TH][k][j];
                sum[T][k][j] += x;
                g[k][j] = e * w[j];
                sg += g[k][j];
                sgh = __builtin_fmaf(g[k][j], h[k][j], sgh);
            }
            if (n > 0) {
                put8<TAIL, RB>(a.dr, r * a.D + c, n, dR[k]);
                if (a.gate_rows && a.dgate) put8<TAIL, OB>(a.dgate, r * a.D + c, n, dg);
            }
        }
        if (a.post) {
            row_sum2<TPR, NTH>(sg, sgh, s, q, turn);
            sg *= inv;
            sgh *= inv;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[k][j] = s1 * (g[k][j] - sg - h[k][j] * sgh);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (li + k * TPR);
            if (D - c > 0) put8<TAIL, OB>(a.d_o, r * a.D + c, D - c, g[k]);
        }
    }
    if (!columns) return;
    const int w = threadIdx.x / TPR;
    float *part = a.part + (int64_t)blockIdx.x * KINDS * a.D;
#pragma unroll
    for (int i = 0; i < KINDS; ++i) {
        if (!has(a, i)) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *(f32x4 *)(acc[w] + 8 * (li + k * TPR) + e) =
                    (f32x4){sum[i][k][e], sum[i][k][e + 1], sum[i][k][e + 2], sum[i][k][e + 3]};
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += NTH) {
            float t = acc[0][c];
#pragma unroll
            for (int j = 1; j < RW; ++j) t += acc[j][c];
            part[(int64_t)i * a.D + c] = t;
        }
        __syncthreads();
    }
}

// Any D: a workgroup its rows one after another, each read three times; a
// thread's columns of the weight gradients are summed in the workgroup's own
// part of the workspace.  Written at the third reading: dr may be dr_out.
template <bool OB, bool RB, bool YB>
__global__ __launch_bounds__(NT) void k_addnorm_bwd_wide(AddNormArgs a) {
    __shared__ float s[2][NT / 64], q[2][NT / 64];
    int turn = 0;
    const bool columns = columns_of(a);
    float *part = a.part + (int64_t)blockIdx.x * KINDS * a.D;
    const float zero[8] = {};
    if (columns)
        for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT)
            for (int i = 0; i < KINDS; ++i) store8n<false>(part, i * (int64_t)a.D + c, a.D - (int)c, zero);
    for (int64_t r = blockIdx.x; r < a.B; r += gridDim.x) {
        float m[2] = {0.f, 0.f}, w[2] = {1.f, 1.f}, sg[2] = {0.f, 0.f}, sgh[2] = {0.f, 0.f};
        if (a.post) {
            m[0] = a.stats[r];
            w[0] = a.stats[a.B + r];
        }
        if (a.norm) {
            m[1] = a.stats[2 * (int64_t)a.B + r];
            w[1] = a.stats[3 * (int64_t)a.B + r];
        }
        for (int pass = a.norm ? 0 : a.post ? 1 : 2; pass < 3; ++pass) {
            float x = 0.f, y = 0.f;
            if (pass == 1 && !a.post) continue;
            for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
                const int n = a.D - (int)c;
                const int64_t i = r * a.D + c;
                float dR[8] = {}, h2[8] = {}, dy[8] = {}, g[8];
                if (a.norm) {
                    load8n<RB>(a.r_out, i, (int)c, a.D, m[1], h2);
                    load8n<YB>(a.dy, i, (int)c, a.D, 0.f, dy);
                    load_w8(a.g2, a.wbf, (int)c, a.D, 1.f, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        h2[j] = j < n ? (h2[j] - m[1]) * w[1] : 0.f;
                        g[j] = j < n ? g[j] * dy[j] : 0.f;
                        if (pass == 0) {
                            x += g[j];
                            y = __builtin_fmaf(g[j], h2[j], y);
                        }
                    }
                }
                if (pass == 0) continue;
                if (a.dr_out) load8n<RB>(a.dr_out, i, (int)c, a.D, 0.f, dR);
                if (a.norm) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dR[j] += w[1] * (g[j] - sg[1] - h2[j] * sgh[1]);
                }
                float o[8], w1[8], b1[8], gate[8], keep[8], e[8], dg[8];
                load8n<OB>(a.o, i, (int)c, a.D, m[0], o);
                load_w8(a.post ? a.g1 : nullptr, a.wbf, (int)c, a.D, 1.f, w1);
                load_w8(a.post ? a.b1 : nullptr, a.wbf, (int)c, a.D, 0.f, b1);
                if (a.gate_rows) load8n<OB>(a.gate, i, (int)c, a.D, 0.f, gate);
                else load_w8(a.gate, a.wbf, (int)c, a.D, 1.f, gate);
                keep8(a.drop, (unsigned)(c >> 3), (unsigned)r, keep);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool in = j < n;
                    o[j] = in ? (o[j] - m[0]) * w[0] : 0.f;
                    const float t = in ? kept(keep[j], a.alpha * dR[j]) : 0.f;
                    const float v = in && keep[j] != 0.f ? gate[j] * t : 0.f;
                    dg[j] = in && keep[j] != 0.f ? t * __builtin_fmaf(o[j], w1[j], b1[j]) : 0.f;
                    e[j] = a.gate_rows ? v : t;
                    keep[j] = keep[j] != 0.f ? o[j] : 0.f;      // a dropped element is not in the sums
                    g[j] = v * w1[j];
                    if (pass == 1) {
                        x += g[j];
                        y = __builtin_fmaf(g[j], o[j], y);
                    }
                }
                if (pass == 1) continue;
                if (a.post) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[j] = w[0] * (g[j] - sg[0] - o[j] * sgh[0]);
                }
                store8n<RB>(a.dr, i, n, dR);
                store8n<OB>(a.d_o, i, n, g);
                if (a.gate_rows && a.dgate) store8n<OB>(a.dgate, i, n, dg);
                if (!columns) continue;
                float p[8];
                auto add = [&](int kind, const float *v, const float *u) {
                    if (!has(a, kind)) return;
                    load8n<false>(part + (int64_t)kind * a.D, c, (int)c, a.D, 0.f, p);
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = u ? __builtin_fmaf(v[j], u[j], p[j]) : p[j] + v[j];
                    store8n<false>(part + (int64_t)kind * a.D, c, n, p);
                };
                add(DYH, dy, h2);
                add(DY, dy, nullptr);
                add(TH, e, keep);
                add(T, e, nullptr);
            }
            if (pass < 2) {
                row_sum2<NT, NT>(x, y, s, q, turn);
                sg[1 - pass] = x / (float)a.D;
                sgh[1 - pass] = y / (float)a.D;
            }
        }
    }
}

// The partial sums of a column added up: 16 waves of 64 columns, a sixteenth
// of the partials each, joined in LDS.  blockIdx.y: y's norm, or the block's side.
__global__ __launch_bounds__(1024) void k_addnorm_wsum(AddNormArgs a, int parts) {
    __shared__ float s[2][16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, first = 2 * blockIdx.y;
    if (!has(a, first) && !has(a, first + 1)) return;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < a.D; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float t = 0.f;
            if (c < a.D && has(a, first + i)) {
                constexpr int U = 8;
                for (int p0 = w; p0 < parts; p0 += 16 * U) {
                    float v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        v[u] = p0 + 16 * u < parts ? a.part[((int64_t)(p0 + 16 * u) * KINDS + first + i) * a.D + c] : 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u) t += v[u];
                }
            }
            s[i][w][lane] = t;
        }
        __syncthreads();
        if (w == 0 && c < a.D) {
            float x = 0.f, y = 0.f;      // with h, without
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x += s[0][i][lane];
                y += s[1][i][lane];
            }
            auto put = [&](float *p, float v) {
                if (p) p[c] = a.accumulate ? p[c] + v : v;
            };
            auto at = [&](const void *p, float none) { return !p ? none : a.wbf ? load1<true>(p, c) : load1<false>(p, c); };
            if (first == 0) {
                put(a.dg2, x);
                put(a.db2, y);
            } else {
                const float gate = a.gate_rows ? 1.f : at(a.gate, 1.f);
                put(a.dg1, gate * x);
                put(a.db1, gate * y);
                if (!a.gate_rows) put((float *)a.dgate, a.post ? at(a.g1, 1.f) * x + (a.b1 ? at(a.b1, 0.f) * y : 0.f) : x);
            }
        }
        __syncthreads();
    }
}

namespace {
// rows of a workgroup at a time; 0: the wide kernel
int bwd_rows(int D) { return D <= 256 ? NB / 16 : D <= 512 ? NB / 32 : D <= 1024 ? NB / 64 : D <= 8192 ? 1 : 0; }
}  // namespace

int addnorm_parts(int B, int D) {
    const int rows = bwd_rows(D);
    const int64_t want = rows ? ((int64_t)B + rows - 1) / rows : B, most = rows ? 512 : 256;
    return (int)(want < most ? want : most);
}

template <bool OB, bool RB, bool YB, bool TAIL>
static hipError_t bwd(const AddNormArgs &a, hipStream_t st) {
    const int parts = addnorm_parts(a.B, a.D);
#define GO(NV, TPR) \
    hipLaunchKernelGGL((k_addnorm_bwd<OB, RB, YB, TAIL, NV, TPR>), dim3(parts), dim3(TPR > NB ? TPR : NB), 0, st, a)
    if (a.D <= 128) GO(1, 16);
    else if (a.D <= 256) GO(2, 16);
    else if (a.D <= 512) GO(2, 32);
    else if (a.D <= 1024) GO(2, 64);
    else if (a.D <= 2048) GO(1, 256);
    else if (a.D <= 4096) GO(1, 512);
    else if (a.D <= 8192) GO(1, 1024);
    else hipLaunchKernelGGL((k_addnorm_bwd_wide<OB, RB, YB>), dim3(parts), dim3(NT), 0, st, a);
#undef GO
    if (columns_of(a)) {
        const int64_t cols = ((int64_t)a.D + 63) / 64;
        hipLaunchKernelGGL(k_addnorm_wsum, dim3((unsigned)(cols < 65536 ? cols : 65536), 2), dim3(1024), 0, st, a, parts);
    }
    return hipGetLastError();
}

hipError_t launch_addnorm_bwd(const AddNormArgs &a, hipStream_t st) { HASTE_PICK_TYPES(bwd, a, st) }

}  // namespace haste
