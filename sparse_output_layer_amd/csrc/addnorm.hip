// addnorm.hip -- a block's output joined to the residual stream between two
// layer norms, in one pass over the rows.
//
//   p  = post ? (o - m1) s1 g1 + b1 : o
//   r' = r + alpha gate drop(p)
//   y  = (r' - m2) s2 g2 + b2
//
// Bound by memory: every element is read once and written once, a row staying
// in the registers of the threads that share it: 65536 x 768 bf16 with dropout 79
// to 83 us, 4.9 to 5.1 TB/s (the weights in registers instead of LDS: 109).
#include "rows.h"

namespace haste {

namespace {
constexpr int NT = 256;
}

// ------------------------------------------------------------------ forward
// NV vectors of eight a thread, TPR threads a row; the next row's vectors are
// loaded while this one is worked on.  The gate of all rows and alpha are
// multiplied into the post norm's weights once a workgroup; where several rows
// share a wave or a workgroup the weights lie in LDS, which leaves registers for
// more waves.  y is made of the sum before it is rounded to the stream's type.
template <bool OB, bool RB, bool YB, bool TAIL, int NV, int TPR>
__global__ __launch_bounds__(TPR > NT ? TPR : NT) void k_addnorm_fwd(AddNormArgs a) {
    constexpr int NTH = TPR > NT ? TPR : NT, RW = NTH / TPR;
    __shared__ float s[2][NTH / 64];
    int turn = 0;
    const int li = threadIdx.x % TPR, tail = tail_of<TAIL, TPR>(a.D);
    constexpr bool LDS = TPR <= 64;
    constexpr int COLS = 8 * NV * TPR;
    __shared__ __attribute__((aligned(16))) float sw[LDS ? 4 * COLS : 4];
    float wr[LDS ? 1 : NV][4][8];        // the thread's: post norm's, with the gate; y's norm's
    auto weights = [&](int c, float (*w)[8]) {
        float g[8];
        load_w8(a.gate_rows ? nullptr : a.gate, a.wbf, c, a.D, 1.f, g);
        load_w8(a.post ? a.g1 : nullptr, a.wbf, c, a.D, 1.f, w[0]);
        load_w8(a.post ? a.b1 : nullptr, a.wbf, c, a.D, 0.f, w[1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[0][j] *= a.alpha * g[j];
            if (a.post) w[1][j] *= a.alpha * g[j];
        }
        load_w8(a.g2, a.wbf, c, a.D, 1.f, w[2]);
        load_w8(a.b2, a.wbf, c, a.D, 0.f, w[3]);
    };
    if (LDS) {
        for (int c = 8 * threadIdx.x; c < COLS; c += 8 * NTH) {
            float w[4][8];
            weights(c, w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *(f32x4 *)(sw + i * COLS + c + e) = (f32x4){w[i][e], w[i][e + 1], w[i][e + 2], w[i][e + 3]};
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) weights(8 * (li + k * TPR), wr[LDS ? 0 : k]);
    }
    // two of the four rows of weights of vector k
    auto pair = [&](int k, int first, int at, float *u, float *v) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            if (LDS) {
                const f32x4 x = *(const f32x4 *)(sw + first * COLS + at + e), y = *(const f32x4 *)(sw + (first + 1) * COLS + at + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[e + j] = x[j];
                    v[e + j] = y[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[e + j] = wr[LDS ? 0 : k][first][e + j];
                    v[e + j] = wr[LDS ? 0 : k][first + 1][e + j];
                }
            }
        }
    };
    Raw8<OB> no[NV], ng[NV];
    Raw8<RB> nr[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (li + k * TPR), D = r < a.B ? a.D : 0;
            const bool t = TAIL && k == tail;
            no[k] = raw8n<OB>(a.o, r * a.D + c, c, D, t);
            nr[k] = raw8n<RB>(a.r, r * a.D + c, c, D, t);
            if (a.gate_rows) ng[k] = raw8n<OB>(a.gate, r * a.D + c, c, D, t);
        }
    };
    const int64_t step = (int64_t)gridDim.x * RW;
    fetch((int64_t)blockIdx.x * RW + threadIdx.x / TPR);
    for (int64_t rb = (int64_t)blockIdx.x * RW; rb < a.B; rb += step) {
        const int64_t r = rb + threadIdx.x / TPR;
        const bool live = r < a.B;                      // all lanes stay for the row sums
        float x[NV][8], t[NV][8], g[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (li + k * TPR);
            const bool e = TAIL && k == tail;
            unpack8n<OB>(no[k], c, a.D, e, x[k]);
            unpack8n<RB>(nr[k], c, a.D, e, t[k]);
            if (a.gate_rows) unpack8n<OB>(ng[k], c, a.D, e, g[k]);
        }
        fetch(r + step);
        float mean = 0.f, rstd = 1.f;
        // mean and deviations of the row in v
        auto norm = [&](float (&v)[NV][8]) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                sum += ((v[k][0] + v[k][1]) + (v[k][2] + v[k][3])) + ((v[k][4] + v[k][5]) + (v[k][6] + v[k][7]));
            mean = row_sum<TPR, NTH>(sum, s, turn) / (float)a.D;
            sum = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int n = a.D - 8 * (li + k * TPR);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[k][j] = j < n ? v[k][j] - mean : 0.f;
                    sum = __builtin_fmaf(v[k][j], v[k][j], sum);
                }
            }
            rstd = 1.0f / sqrtf(row_sum<TPR, NTH>(sum, s, turn) / (float)a.D + a.eps);
        };
        if (a.post) {
            norm(x);
            if (a.stats && live && li == 0) {
                a.stats[r] = mean;
                a.stats[a.B + r] = rstd;
            }
        }
        const int lw = LDS ? opaque_index(li) : li;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = li + k * TPR, c = 8 * v;
            if (c < a.D) {
                float ca[8], cb[8];
                pair(k, 0, 8 * (lw + k * TPR), ca, cb);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = __builtin_fmaf(x[k][j] * rstd, ca[j], cb[j]);
                if (a.gate_rows) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[k][j] *= g[k][j];
                }
                if (a.drop.thr) drop8(a.drop, (unsigned)v, (unsigned)r, x[k]);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[k][j] = TAIL && j >= a.D - c ? 0.f : t[k][j] + x[k][j];
                if (live) put8<TAIL, RB>(a.r_out, r * a.D + c, a.D - c, t[k]);
            }
        }
        if (!a.y) continue;
        norm(t);
        if (!live) continue;
        if (a.stats && li == 0) {
            a.stats[2 * (int64_t)a.B + r] = mean;
            a.stats[3 * (int64_t)a.B + r] = rstd;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (li + k * TPR);
            if (c >= a.D) continue;
            float g2[8], b2[8];
            pair(k, 2, 8 * (lw + k * TPR), g2, b2);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[k][j] = __builtin_fmaf(t[k][j] * rstd, g2[j], b2[j]);
            put8<TAIL, YB>(a.y, r * a.D + c, a.D - c, t[k]);
        }
    }
}

// Any D: a workgroup a row, its sums from further readings (of L2); nothing is
// written before the last, so that r_out may be r.
template <bool OB, bool RB, bool YB>
__global__ __launch_bounds__(NT) void k_addnorm_fwd_wide(AddNormArgs a) {
    __shared__ float s[2][NT / 64];
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.B; r += gridDim.x) {
        float m[2] = {0.f, 0.f}, q[2] = {1.f, 1.f};
        // eight values of o, or of the joined stream
        auto block = [&](int64_t c, float *x) { load8n<OB>(a.o, r * a.D + c, (int)c, a.D, m[0], x); };
        auto joined = [&](int64_t c, float *t) {
            float x[8], w[8];
            block(c, x);
            load_w8(a.post ? a.g1 : nullptr, a.wbf, (int)c, a.D, 1.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (x[j] - m[0]) * q[0] * w[j];
            load_w8(a.post ? a.b1 : nullptr, a.wbf, (int)c, a.D, 0.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] += w[j];
            if (a.gate_rows) load8n<OB>(a.gate, r * a.D + c, (int)c, a.D, 0.f, w);
            else load_w8(a.gate, a.wbf, (int)c, a.D, 1.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= a.alpha * w[j];
            if (a.drop.thr) drop8(a.drop, (unsigned)(c >> 3), (unsigned)r, x);
            load8n<RB>(a.r, r * a.D + c, (int)c, a.D, 0.f, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] += x[j];
        };
        for (int k = a.post ? 0 : 1; k < (a.y ? 2 : 1); ++k) {
            float sum = 0.f, v[8];
            for (int pass = 0; pass < 2; ++pass) {
                sum = 0.f;
                for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
                    if (k) joined(c, v);
                    else load8n<OB>(a.o, r * a.D + c, (int)c, a.D, 0.f, v);
                    const int n = a.D - (int)c;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float d = pass ? v[j] - m[k] : v[j];
                        if (j < n) sum = pass ? __builtin_fmaf(d, d, sum) : sum + d;
                    }
                }
                sum = row_sum<NT, NT>(sum, s, turn) / (float)a.D;
                // m[0] and q[0] are used by joined() only once both are known
                if (pass == 0) m[k] = sum;
                else q[k] = 1.0f / sqrtf(sum + a.eps);
            }
            if (a.stats && threadIdx.x == 0) {
                a.stats[2 * k * (int64_t)a.B + r] = m[k];
                a.stats[(2 * k + 1) * (int64_t)a.B + r] = q[k];
            }
        }
        for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
            float t[8], w[8];
            joined(c, t);
            store8n<RB>(a.r_out, r * a.D + c, a.D - (int)c, t);
            if (!a.y) continue;
            load_w8(a.g2, a.wbf, (int)c, a.D, 1.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = (t[j] - m[1]) * q[1] * w[j];
            load_w8(a.b2, a.wbf, (int)c, a.D, 0.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] += w[j];
            store8n<YB>(a.y, r * a.D + c, a.D - (int)c, t);
        }
    }
}

template <bool OB, bool RB, bool YB, bool TAIL>
static hipError_t fwd(const AddNormArgs &a, hipStream_t st) {
    auto grid = [&](int rows, int64_t most) {
        const int64_t want = ((int64_t)a.B + rows - 1) / rows;
        return dim3((unsigned)(want < most ? want : most));
    };
#define GO(NV, TPR) \
    hipLaunchKernelGGL((k_addnorm_fwd<OB, RB, YB, TAIL, NV, TPR>), grid(TPR > NT ? 1 : NT / TPR, 2048), dim3(TPR > NT ? TPR : NT), 0, st, a)
    if (a.D <= 128) GO(1, 16);
    else if (a.D <= 256) GO(2, 16);
    else if (a.D <= 512) GO(2, 32);
    else if (a.D <= 768) GO(3, 32);
    else if (a.D <= 1024) GO(2, 64);
    else if (a.D <= 2048) GO(1, 256);
    else if (a.D <= 4096) GO(2, 256);
    else if (a.D <= 8192) GO(2, 512);
    else hipLaunchKernelGGL((k_addnorm_fwd_wide<OB, RB, YB>), grid(1, 4096), dim3(NT), 0, st, a);
#undef GO
    return hipGetLastError();
}

hipError_t launch_addnorm_fwd(const AddNormArgs &a, hipStream_t st) { HASTE_PICK_TYPES(fwd, a, st) }

}  // namespace haste
