// norm.hip -- layer norm (forward, backward, weight gradient) and dropout
// from a counter-based generator.
#include "elem.h"

namespace haste {

namespace {

constexpr int NT = 256;

// Sum over the workgroup of NT threads, in a fixed order; every thread gets
// it.  s: LDS room for NT / 64 floats.
__device__ __forceinline__ float block_sum(float v, float *s) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < NT / 64; ++i) t += s[i];
    return t;
}

// one element's kept value (dropped: 0)
__device__ __forceinline__ float drop1(const DropArgs &d, int c, int r, float v) {
    if (d.thr == 0) return v;
    return (drop_keep8(d, (unsigned)c >> 3, (unsigned)r) >> (c & 7)) & 1u ? v * d.scale : 0.f;
}

}  // namespace

// ---------------------------------------------------------------- dropout
template <bool XB, bool YB>
__global__ __launch_bounds__(NT) void k_dropout(int B, int D, const void *x, DropArgs d, void *y) {
    const int nv = (D + 7) / 8;
    const int64_t total = (int64_t)B * nv;
    for (int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x; t < total; t += (int64_t)gridDim.x * NT) {
        const int64_t r = t / nv;
        const int v = (int)(t - r * nv);
        const unsigned keep = d.thr ? drop_keep8(d, (unsigned)v, (unsigned)r) : 0xffu;
        for (int j = 0; j < 8 && 8 * v + j < D; ++j) {
            const int64_t i = r * D + 8 * (int64_t)v + j;
            const float a = load1<XB>(x, i);
            store1<YB>(y, i, (keep >> j) & 1u ? a * d.scale : 0.f);
        }
    }
}

hipError_t launch_dropout(int B, int D, bool xbf, bool ybf, const void *x, const DropArgs &dr, void *y,
                          hipStream_t st) {
    const int64_t total = (int64_t)B * ((D + 7) / 8);
    const int64_t want = (total + NT - 1) / NT;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536));
#define GO(X, Y) hipLaunchKernelGGL((k_dropout<X, Y>), grid, dim3(NT), 0, st, B, D, x, dr, y)
    if (xbf && ybf) GO(true, true);
    else if (xbf) GO(true, false);
    else if (ybf) GO(false, true);
    else GO(false, false);
#undef GO
    return hipGetLastError();
}

// ------------------------------------------------------------- layer norm
template <bool XB, bool YB>
__global__ __launch_bounds__(NT) void k_norm_fwd(NormArgs a) {
    __shared__ float s[NT / 64];
    for (int64_t r = blockIdx.x; r < a.B; r += gridDim.x) {
        const int64_t o = r * a.ldx;
        float v = 0.f;
        for (int c = threadIdx.x; c < a.D; c += NT) v += load1<XB>(a.x, o + c);
        const float mean = block_sum(v, s) / (float)a.D;
        v = 0.f;
        for (int c = threadIdx.x; c < a.D; c += NT) {
            const float d = load1<XB>(a.x, o + c) - mean;
            v += d * d;
        }
        const float rstd = 1.0f / sqrtf(block_sum(v, s) / (float)a.D + a.eps);
        for (int c = threadIdx.x; c < a.D; c += NT) {
            float y = (load1<XB>(a.x, o + c) - mean) * rstd;
            if (a.gamma) y *= a.wbf ? load1<true>(a.gamma, c) : load1<false>(a.gamma, c);
            if (a.beta) y += a.wbf ? load1<true>(a.beta, c) : load1<false>(a.beta, c);
            store1<YB>(a.y, r * a.D + c, drop1(a.drop, c, (int)r, y));
        }
        if (a.mean && threadIdx.x == 0) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
    }
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)(a.B < 65536 ? a.B : 65536));
#define GO(X, Y) hipLaunchKernelGGL((k_norm_fwd<X, Y>), grid, dim3(NT), 0, st, a)
    if (a.xbf && a.ybf) GO(true, true);
    else if (a.xbf) GO(true, false);
    else if (a.ybf) GO(false, true);
    else GO(false, false);
#undef GO
    return hipGetLastError();
}

template <bool XB, bool YB>
__global__ __launch_bounds__(NT) void k_norm_bwd(NormArgs a) {
    __shared__ float s[NT / 64];
    for (int64_t r = blockIdx.x; r < a.B; r += gridDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float sg = 0.f, sgh = 0.f;
        for (int c = threadIdx.x; c < a.D; c += NT) {
            const float h = (load1<XB>(a.x, r * a.ldx + c) - mean) * rstd;
            float g = drop1(a.drop, c, (int)r, load1<YB>(a.dy, r * a.D + c));
            if (a.gamma) g *= a.wbf ? load1<true>(a.gamma, c) : load1<false>(a.gamma, c);
            sg += g;
            sgh += g * h;
        }
        sg = block_sum(sg, s) / (float)a.D;
        sgh = block_sum(sgh, s) / (float)a.D;
        for (int c = threadIdx.x; c < a.D; c += NT) {
            const float h = (load1<XB>(a.x, r * a.ldx + c) - mean) * rstd;
            float g = drop1(a.drop, c, (int)r, load1<YB>(a.dy, r * a.D + c));
            if (a.gamma) g *= a.wbf ? load1<true>(a.gamma, c) : load1<false>(a.gamma, c);
            store1<XB>(a.dx, r * a.lddx + c, rstd * (g - sg - h * sgh));
        }
    }
}

// part[p][0..1][c]: the sums of a * h and a over the rows p, p + parts, ...
template <bool XB, bool YB>
__global__ __launch_bounds__(NT) void k_norm_wgrad(NormArgs a) {
    const int c = blockIdx.x * NT + threadIdx.x, parts = gridDim.y;
    if (c >= a.D) return;
    float dg = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.B; r += parts) {
        const float h = (load1<XB>(a.x, r * a.ldx + c) - a.mean[r]) * a.rstd[r];
        const float v = drop1(a.drop, c, (int)r, load1<YB>(a.dy, r * a.D + c));
        dg += v * h;
        db += v;
    }
    a.part[((int64_t)blockIdx.y * 2) * a.D + c] = dg;
    a.part[((int64_t)blockIdx.y * 2 + 1) * a.D + c] = db;
}

__global__ __launch_bounds__(NT) void k_norm_wsum(NormArgs a, int parts) {
    const int c = blockIdx.x * NT + threadIdx.x;
    if (c >= a.D) return;
    float dg = 0.f, db = 0.f;
    for (int p = 0; p < parts; ++p) {
        dg += a.part[((int64_t)p * 2) * a.D + c];
        db += a.part[((int64_t)p * 2 + 1) * a.D + c];
    }
    if (a.dgamma) a.dgamma[c] = a.accumulate ? a.dgamma[c] + dg : dg;
    if (a.dbeta) a.dbeta[c] = a.accumulate ? a.dbeta[c] + db : db;
}

int norm_parts(int B, int D) { return B < 256 ? B : 256; }

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)(a.B < 65536 ? a.B : 65536));
    const int parts = norm_parts(a.B, a.D);
    const bool w = a.dgamma || a.dbeta;
#define GO(X, Y)                                                                                          \
    {                                                                                                     \
        hipLaunchKernelGGL((k_norm_bwd<X, Y>), grid, dim3(NT), 0, st, a);                                 \
        if (w) hipLaunchKernelGGL((k_norm_wgrad<X, Y>), dim3((a.D + NT - 1) / NT, parts), dim3(NT), 0, st, a); \
    }
    if (a.xbf && a.ybf) GO(true, true)
    else if (a.xbf) GO(true, false)
    else if (a.ybf) GO(false, true)
    else GO(false, false)
#undef GO
    if (w) hipLaunchKernelGGL(k_norm_wsum, dim3((a.D + NT - 1) / NT), dim3(NT), 0, st, a, parts);
    return hipGetLastError();
}

}  // namespace haste
