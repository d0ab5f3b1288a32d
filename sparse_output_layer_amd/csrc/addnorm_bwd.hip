// addnorm_bwd.hip -- gradients of a block's output joined to the residual
// stream between two layer norms (addnorm.hip), in one pass over the rows:
//
//   h2 = (r' - m2) s2, u = dy g2, dR = dr' + s2 (u - mean(u) - h2 mean(u h2))
//   dr = dR, a = drop(alpha gate dR), dgate = alpha dR drop(p)
//   h1 = (o - m1) s1, v = a g1, do = post ? s1 (v - mean(v) - h1 mean(v h1)) : a
//   dg2 = sum dy h2, db2 = sum dy, dg1 = sum a h1, db1 = sum a   (over the rows)
//
// Bound by memory: r', dy, dr', o in, dr and do out, a row staying in the
// registers of the threads that share it.  The weight gradients (five rows of
// D at most) are summed over a workgroup's rows in registers, its threads'
// sums joined in LDS, and the workgroups' partial sums added up by a second
// launch, all in a fixed order.
#include "rows.h"

namespace haste {

namespace {

constexpr int NT = 256;
constexpr int NB = 512;       // threads of a workgroup whose rows are shorter
enum { DG2, DB2, DG1, DB1, DGATE, KINDS };

// which partial sums a call has
__device__ __forceinline__ bool has(const AddNormArgs &a, int kind) {
    switch (kind) {
    case DG2: return a.dg2;
    case DB2: return a.db2;
    case DG1: return a.dg1;
    case DB1: return a.db1;
    default: return a.dgate && !a.gate_rows;
    }
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
__global__ __launch_bounds__(TPR > NB ? TPR : NB, TPR > NB ? 4 : 2) void k_addnorm_bwd(AddNormArgs a) {
    constexpr int NTH = TPR > NB ? TPR : NB, RW = NTH / TPR;
    __shared__ float s[2][NTH / 64], q[2][NTH / 64];
    __shared__ __attribute__((aligned(16))) float acc[RW][8 * NV * TPR];
    int turn = 0;
    const int li = threadIdx.x % TPR, tail = tail_of<TAIL, TPR>(a.D);
    const bool columns = a.dg1 || a.db1 || a.dg2 || a.db2 || (a.dgate && !a.gate_rows);
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
        const int D = live ? a.D : 0;
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
                load_w8(a.g2, a.wbf, c, a.D, 1.f, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[k][j] = (TAIL ? j < n : n > 0) ? (h[k][j] - mean) * rstd : 0.f;
                    sum[DG2][k][j] = __builtin_fmaf(g[k][j], h[k][j], sum[DG2][k][j]);
                    sum[DB2][k][j] += g[k][j];
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
            else load_w8(a.gate, a.wbf, c, a.D, 1.f, gate);
            load_w8(a.post ? a.g1 : nullptr, a.wbf, c, a.D, 1.f, w);
            load_w8(a.post ? a.b1 : nullptr, a.wbf, c, a.D, 0.f, b1);
            keep8(a.drop, (unsigned)v, (unsigned)r, keep);
            float dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = TAIL ? j < n : n > 0;
                h[k][j] = in ? (h[k][j] - m1) * s1 : 0.f;
                const float t = in ? a.alpha * dR[k][j] : 0.f;
                const float e = in ? kept(keep[j], gate[j] * t) : 0.f;
                dg[j] = in ? kept(keep[j], t * __builtin_fmaf(h[k][j], w[j], b1[j])) : 0.f;
                sum[DGATE][k][j] += dg[j];
                sum[DG1][k][j] = __builtin_fmaf(e, h[k][j], sum[DG1][k][j]);
                sum[DB1][k][j] += e;
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
    const bool columns = a.dg1 || a.db1 || a.dg2 || a.db2 || (a.dgate && !a.gate_rows);
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
                    const float t = in ? a.alpha * dR[j] : 0.f;
                    e[j] = in ? kept(keep[j], gate[j] * t) : 0.f;
                    dg[j] = in ? kept(keep[j], t * __builtin_fmaf(o[j], w1[j], b1[j])) : 0.f;
                    g[j] = e[j] * w1[j];
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
                add(DG2, dy, h2);
                add(DB2, dy, nullptr);
                add(DG1, e, o);
                add(DB1, e, nullptr);
                add(DGATE, dg, nullptr);
            }
            if (pass < 2) {
                row_sum2<NT, NT>(x, y, s, q, turn);
                sg[1 - pass] = x / (float)a.D;
                sgh[1 - pass] = y / (float)a.D;
            }
        }
    }
}

// The partial sums of a column of one kind added up: 16 waves of 64 columns, a
// sixteenth of the partials each, joined in LDS.
__global__ __launch_bounds__(1024) void k_addnorm_wsum(AddNormArgs a, int parts) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, kind = blockIdx.y;
    if (!has(a, kind)) return;
    float *out = kind == DG2 ? a.dg2 : kind == DB2 ? a.db2 : kind == DG1 ? a.dg1 : kind == DB1 ? a.db1 : (float *)a.dgate;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < a.D; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float t = 0.f;
        if (c < a.D) {
            constexpr int U = 8;
            for (int p0 = w; p0 < parts; p0 += 16 * U) {
                float v[U];
#pragma unroll
                for (int i = 0; i < U; ++i)
                    v[i] = p0 + 16 * i < parts ? a.part[((int64_t)(p0 + 16 * i) * KINDS + kind) * a.D + c] : 0.f;
#pragma unroll
                for (int i = 0; i < U; ++i) t += v[i];
            }
        }
        s[w][lane] = t;
        __syncthreads();
        if (w == 0 && c < a.D) {
            t = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) t += s[i][lane];
            out[c] = a.accumulate ? out[c] + t : t;
        }
        __syncthreads();
    }
}

namespace {
// rows of a workgroup at a time; 0: the wide kernel
int bwd_rows(int D) { return D <= 256 ? NB / 16 : D <= 1024 ? NB / 64 : D <= 2048 ? NB / 256 : D <= 8192 ? 1 : 0; }
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
    else if (a.D <= 512) GO(1, 64);
    else if (a.D <= 1024) GO(2, 64);
    else if (a.D <= 2048) GO(1, 256);
    else if (a.D <= 4096) GO(1, 512);
    else if (a.D <= 8192) GO(1, 1024);
    else hipLaunchKernelGGL((k_addnorm_bwd_wide<OB, RB, YB>), dim3(parts), dim3(NT), 0, st, a);
#undef GO
    if (a.dg1 || a.db1 || a.dg2 || a.db2 || (a.dgate && !a.gate_rows)) {
        const int64_t cols = ((int64_t)a.D + 63) / 64;
        hipLaunchKernelGGL(k_addnorm_wsum, dim3((unsigned)(cols < 65536 ? cols : 65536), KINDS), dim3(1024), 0, st, a, parts);
    }
    return hipGetLastError();
}

hipError_t launch_addnorm_bwd(const AddNormArgs &a, hipStream_t st) { HASTE_PICK_TYPES(bwd, a, st) }

}  // namespace haste
