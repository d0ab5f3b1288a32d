// head_i8.hip -- rows in 8-bit integers with one scale each, and the head's
// logits from them.
#include "elem.h"

namespace haste {

namespace {
constexpr int NT = 256;
// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }
}  // namespace

template <bool BF>
__global__ __launch_bounds__(NT) void k_quantize_rows(int rows, int D, int64_t ldx, const void *x, int8_t *q,
                                                      float *scale) {
    __shared__ float s[NT / 64];
    const int D64 = (D + 63) / 64 * 64;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        float m = 0.f;
        for (int c = threadIdx.x; c < D; c += NT) m = max_nan(m, fabsf(load1<BF>(x, r * ldx + c)));
        for (int o = 32; o > 0; o >>= 1) m = max_nan(m, __shfl_xor(m, o, 64));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
        __syncthreads();
        m = s[0];
        for (int i = 1; i < NT / 64; ++i) m = max_nan(m, s[i]);
        const float sc = m / 127.0f;
        for (int c = threadIdx.x; c < D64; c += NT) {
            // zeros in a row whose scale is no number, so that its logits are NaN
            float t = c < D && sc > 0.f && sc < __builtin_inff() ? rintf(load1<BF>(x, r * ldx + c) / sc) : 0.f;
            t = fminf(fmaxf(t, -127.f), 127.f);
            q[r * D64 + c] = (int8_t)(int)t;
        }
        if (threadIdx.x == 0) scale[r] = sc;
    }
}

hipError_t launch_quantize_rows(int rows, int D, bool bf, int64_t ldx, const void *x, int8_t *q, float *scale,
                                hipStream_t st) {
    const dim3 grid((unsigned)(rows < 65536 ? rows : 65536));
    if (bf) hipLaunchKernelGGL(k_quantize_rows<true>, grid, dim3(NT), 0, st, rows, D, ldx, x, q, scale);
    else hipLaunchKernelGGL(k_quantize_rows<false>, grid, dim3(NT), 0, st, rows, D, ldx, x, q, scale);
    return hipGetLastError();
}

template <bool ZB>
__global__ __launch_bounds__(NT) void k_gemm_i8(int M, int N, int K64, const int8_t *A, const float *as,
                                                const int8_t *Bm, const float *bs, void *Z) {
    const int64_t total = (int64_t)M * N;
    for (int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x; t < total; t += (int64_t)gridDim.x * NT) {
        const int64_t m = t / N, n = t - m * N;
        const int *pa = (const int *)(A + m * K64), *pb = (const int *)(Bm + n * K64);
        int acc = 0;
        for (int k = 0; k < K64 / 4; ++k) acc = __builtin_amdgcn_sdot4(pa[k], pb[k], acc, false);
        store1<ZB>(Z, t, (float)acc * as[m] * bs[n]);
    }
}

hipError_t launch_gemm_i8(int M, int N, int K, const int8_t *A, const float *as, const int8_t *Bm, const float *bs,
                          void *Z, bool zbf, hipStream_t st) {
    const int64_t want = ((int64_t)M * N + NT - 1) / NT;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536));
    const int K64 = (K + 63) / 64 * 64;
    if (zbf) hipLaunchKernelGGL(k_gemm_i8<true>, grid, dim3(NT), 0, st, M, N, K64, A, as, Bm, bs, Z);
    else hipLaunchKernelGGL(k_gemm_i8<false>, grid, dim3(NT), 0, st, M, N, K64, A, as, Bm, bs, Z);
    return hipGetLastError();
}

}  // namespace haste
