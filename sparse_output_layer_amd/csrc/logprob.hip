// logprob.hip -- softmax statistics over head and tail logits: log
// probabilities of given labels, entropy, top alternatives, and the gradient.
#include "elem.h"

namespace haste {

namespace {

constexpr int NT = 256;
constexpr int CHUNK = 8192;   // logits of a row per workgroup

// A candidate's key: larger is better (value descending, then label
// ascending); 0: none.
__device__ __forceinline__ unsigned long long cand_key(float v, unsigned label) {
    return ((unsigned long long)f32_order_key(v) << 32) | (0xffffffffu - label);
}
__device__ __forceinline__ bool is_cand(float v) { return v > -__builtin_inff(); }   // false for NaN

__device__ __forceinline__ unsigned long long block_max(unsigned long long k, unsigned long long *s) {
    for (int o = 32; o > 0; o >>= 1) {
        const unsigned long long t = __shfl_xor(k, o, 64);
        k = t > k ? t : k;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = k;
    __syncthreads();
    for (int i = 0; i < NT / 64; ++i) k = s[i] > k ? s[i] : k;
    return k;
}

// Softmax statistics: maximum m, S = sum e^(z - m), T = sum e^(z - m) (z - m).
// S = 0: no logit above -inf yet (m = -inf).
struct Stat {
    float m, S, T;
};
// One logit.  z - m of a masked logit is -inf, its e is 0 and its part in T
// is 0 by the clamp; NaN and +inf end as NaN in S.
__device__ __forceinline__ void stat_add(Stat &s, float z) {
    if (z == -__builtin_inff()) return;
    if (z > s.m) {
        const float d = s.m - z;   // <= 0, -inf at the first logit
        const float f = s.S == 0.f ? 0.f : __expf(d);
        s.T = s.S == 0.f ? 0.f : f * (s.T + fmaxf(d, -1e4f) * s.S);
        s.S *= f;
        s.m = z;
    }
    const float v = z - s.m, e = __expf(v);
    s.S += e;
    s.T += e * fmaxf(v, -1e4f);
}
__device__ __forceinline__ Stat stat_join(const Stat &a, const Stat &b) {
    if (a.S == 0.f) return b;
    if (b.S == 0.f) return a;
    const float m = fmaxf(a.m, b.m);
    const float da = a.m - m, db = b.m - m, fa = __expf(da), fb = __expf(db);
    Stat r;
    r.m = m;
    r.S = a.S * fa + b.S * fb;
    r.T = fa * (a.T + fmaxf(da, -1e4f) * a.S) + fb * (b.T + fmaxf(db, -1e4f) * b.S);
    return r;
}
__device__ __forceinline__ Stat block_join(Stat v, Stat *s) {
    for (int o = 1; o < 64; o <<= 1) {
        Stat t;
        t.m = __shfl_xor(v.m, o, 64);
        t.S = __shfl_xor(v.S, o, 64);
        t.T = __shfl_xor(v.T, o, 64);
        v = stat_join(v, t);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    Stat r = s[0];
    for (int i = 1; i < NT / 64; ++i) r = stat_join(r, s[i]);
    return r;
}

__host__ __device__ inline int64_t n_chunks(int64_t n) { return (n + CHUNK - 1) / CHUNK; }

// workspace: stats (B x chunks), keys (B x chunks x K), row losses (B)
struct Ws {
    Stat *stat;
    unsigned long long *key;
    float *loss;
};
__host__ __device__ inline Ws ws_map(const LogprobArgs &a) {
    const int64_t nc = n_chunks(a.n[0]) + n_chunks(a.n[1]);
    Ws w;
    w.key = (unsigned long long *)a.ws;
    w.stat = (Stat *)(w.key + (int64_t)a.B * nc * a.K);
    w.loss = (float *)(w.stat + (int64_t)a.B * nc);
    return w;
}

// chunk index -> part, its first label of the part and its length
__device__ __forceinline__ int chunk_of(const LogprobArgs &a, int64_t c, int64_t *j0, int *len) {
    const int64_t n0 = n_chunks(a.n[0]);
    const int p = c < n0 ? 0 : 1;
    *j0 = (p ? c - n0 : c) * CHUNK;
    const int64_t left = a.n[p] - *j0;
    *len = left < CHUNK ? (int)left : CHUNK;
    return p;
}

}  // namespace

size_t logprob_ws_bytes(int B, int64_t H, int64_t L, bool bf, int K) {
    const int64_t nc = n_chunks(H) + n_chunks(L);
    return (size_t)B * nc * K * 8 + (size_t)B * nc * sizeof(Stat) + (size_t)B * 4;
}

template <bool BF>
__global__ __launch_bounds__(NT) void k_lp_stats(LogprobArgs a, int64_t nc) {
    __shared__ Stat ss[NT / 64];
    __shared__ unsigned long long sk[NT / 64];
    const int64_t item = blockIdx.x, b = item / nc, c = item - b * nc;
    int64_t j0;
    int len;
    const int p = chunk_of(a, c, &j0, &len);
    const int64_t base = b * a.ld[p] + j0;
    const Ws w = ws_map(a);
    Stat st = {-__builtin_inff(), 0.f, 0.f};
    for (int i = threadIdx.x; i < len; i += NT) stat_add(st, load1<BF>(a.z[p], base + i));
    st = block_join(st, ss);
    if (threadIdx.x == 0) w.stat[item] = st;
    const unsigned l0 = (unsigned)((p ? a.n[0] : 0) + j0);
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.K; ++k) {
        unsigned long long best = 0;
        for (int i = threadIdx.x; i < len; i += NT) {
            const float z = load1<BF>(a.z[p], base + i);
            if (!is_cand(z)) continue;
            const unsigned long long key = cand_key(z, l0 + i);
            if (key < last && key > best) best = key;
        }
        best = block_max(best, sk);
        if (threadIdx.x == 0) w.key[item * a.K + k] = best;
        last = best;
    }
}

template <bool BF>
__global__ __launch_bounds__(NT) void k_lp_rows(LogprobArgs a, int64_t nc) {
    __shared__ Stat ss[NT / 64];
    __shared__ unsigned long long sk[NT / 64];
    __shared__ float sl[NT / 64];
    const int64_t b = blockIdx.x;
    const Ws w = ws_map(a);
    Stat st = {-__builtin_inff(), 0.f, 0.f};
    for (int64_t c = threadIdx.x; c < nc; c += NT) st = stat_join(st, w.stat[b * nc + c]);
    st = block_join(st, ss);
    const bool none = st.S == 0.f;
    const float lse = none ? -__builtin_inff() : st.m + logf(st.S);
    if (threadIdx.x == 0) {
        a.lse[b] = lse;
        if (a.entropy) a.entropy[b] = none ? 0.f : logf(st.S) - st.T / st.S;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.K; ++k) {
        unsigned long long best = 0;
        for (int64_t i = threadIdx.x; i < nc * a.K; i += NT) {
            const unsigned long long key = w.key[b * nc * a.K + i];
            if (key < last && key > best) best = key;
        }
        best = block_max(best, sk);
        last = best;
        if (threadIdx.x == 0) {
            a.top_v[b * a.K + k] = best ? f32_from_order_key((unsigned)(best >> 32)) - lse : -__builtin_inff();
            a.top_i[b * a.K + k] = best ? (int32_t)(a.off + (0xffffffffu - (unsigned)best)) : -1;
        }
    }
    if (!a.row_ptr || (!a.logp && !a.loss)) return;
    const int e0 = max(a.row_ptr[b], 0), e1 = min(a.row_ptr[b + 1], a.nnz);
    float sum = 0.f;
    for (int e = e0 + threadIdx.x; e < e1; e += NT) {
        const int64_t j = (int64_t)a.labels[e] - a.off;
        float lp = -__builtin_inff();
        if (j >= 0 && j < a.n[0] + a.n[1]) {
            const int p = j >= a.n[0];
            if (!none) lp = load1<BF>(a.z[p], b * a.ld[p] + (p ? j - a.n[0] : j)) - lse;
            sum -= lp;
        }
        if (a.logp) a.logp[e] = lp;
    }
    if (!a.loss) return;
    sum = wave_sum(sum);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sl[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.f;
        for (int i = 0; i < NT / 64; ++i) t += sl[i];
        w.loss[b] = t;
    }
}

// *loss += s * the sum of the rows' losses, in a fixed order
__global__ __launch_bounds__(NT) void k_lp_loss(LogprobArgs a) {
    __shared__ float sl[NT / 64];
    const Ws w = ws_map(a);
    float t = 0.f;
    for (int b = threadIdx.x; b < a.B; b += NT) t += w.loss[b];
    t = wave_sum(t);
    if ((threadIdx.x & 63) == 0) sl[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        t = 0.f;
        for (int i = 0; i < NT / 64; ++i) t += sl[i];
        *a.loss += a.s * t;
    }
}

hipError_t launch_logprob_fwd(const LogprobArgs &a, hipStream_t st) {
    const int64_t nc = n_chunks(a.n[0]) + n_chunks(a.n[1]);
    const int64_t items = nc * a.B;
    if (items * NT > (int64_t)UINT32_MAX) return hipErrorInvalidValue;   // one launch's threads
    if (a.bf) {
        hipLaunchKernelGGL(k_lp_stats<true>, dim3((unsigned)items), dim3(NT), 0, st, a, nc);
        hipLaunchKernelGGL(k_lp_rows<true>, dim3(a.B), dim3(NT), 0, st, a, nc);
    } else {
        hipLaunchKernelGGL(k_lp_stats<false>, dim3((unsigned)items), dim3(NT), 0, st, a, nc);
        hipLaunchKernelGGL(k_lp_rows<false>, dim3(a.B), dim3(NT), 0, st, a, nc);
    }
    if (a.loss) hipLaunchKernelGGL(k_lp_loss, dim3(1), dim3(NT), 0, st, a);
    return hipGetLastError();
}

// dz of one logit, before its labels' own gradients: -p (G + n (log p + H))
__device__ __forceinline__ float dz_dense(float z, float lse, float G, float n, float H) {
    const float lp = z - lse, p = __expf(lp);
    return -p * (G + n * (fmaxf(lp, -1e4f) + H));
}

template <bool BF>
__global__ __launch_bounds__(NT) void k_lp_bwd(LogprobArgs a, int64_t nc) {
    const int64_t item = blockIdx.x, b = item / nc, c = item - b * nc;
    int64_t j0;
    int len;
    const int p = chunk_of(a, c, &j0, &len);
    const int64_t base = b * a.ld[p] + j0, obase = b * a.n[p] + j0;
    const float lse = a.lse[b];
    const bool none = lse == -__builtin_inff();
    const float n = a.dent ? a.dent[b] : 0.f, H = a.dent ? a.entropy[b] : 0.f;
    int e0 = 0, e1 = 0;
    if (a.row_ptr) {
        e0 = max(a.row_ptr[b], 0);
        e1 = min(a.row_ptr[b + 1], a.nnz);
    }
    const int64_t N = a.n[0] + a.n[1];
    float G = 0.f;
    for (int e = e0; e < e1; ++e) {
        const int64_t j = (int64_t)a.labels[e] - a.off;
        if (j >= 0 && j < N) G += a.dlogp ? a.dlogp[e] : -a.s;
    }
    for (int i = threadIdx.x; i < len; i += NT)
        store1<BF>(a.dz[p], obase + i, none ? 0.f : dz_dense(load1<BF>(a.z[p], base + i), lse, G, n, H));
    if (none) return;
    // the chunk's given labels, each by the thread of its first entry
    __syncthreads();
    const int64_t l0 = (p ? a.n[0] : 0) + j0;
    for (int e = e0 + threadIdx.x; e < e1; e += NT) {
        const int32_t id = a.labels[e];
        const int64_t i = (int64_t)id - a.off - l0;
        if (i < 0 || i >= len) continue;
        float g = 0.f;
        bool first = true;
        for (int f = e0; f < e1; ++f) {
            if (a.labels[f] != id) continue;
            if (f < e) first = false;
            g += a.dlogp ? a.dlogp[f] : -a.s;
        }
        if (first) store1<BF>(a.dz[p], obase + i, g + dz_dense(load1<BF>(a.z[p], base + i), lse, G, n, H));
    }
}

hipError_t launch_logprob_bwd(const LogprobArgs &a, hipStream_t st) {
    const int64_t nc = n_chunks(a.n[0]) + n_chunks(a.n[1]);
    const int64_t items = nc * a.B;
    if (items * NT > (int64_t)UINT32_MAX) return hipErrorInvalidValue;   // one launch's threads
    if (a.bf) hipLaunchKernelGGL(k_lp_bwd<true>, dim3((unsigned)items), dim3(NT), 0, st, a, nc);
    else hipLaunchKernelGGL(k_lp_bwd<false>, dim3((unsigned)items), dim3(NT), 0, st, a, nc);
    return hipGetLastError();
}

}  // namespace haste
