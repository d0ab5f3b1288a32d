// logprob.hip -- softmax statistics over head and tail logits: log
// probabilities of given labels, entropy, top alternatives, and the gradient.
//
// One reading of the logits.  A row's head and tail parts are cut into chunks
// of at most 64 KB; a workgroup loads its chunk into registers and forms
//   M = max z, S = sum e^(z - M), T = sum e^(z - M) (z - M)
// and the chunk's K best logits; a second kernel joins a row's chunks,
//   S = sum_c S_c e^(M_c - M),  T = sum_c e^(M_c - M) (T_c + (M_c - M) S_c),
//   lse = M + log S,  entropy = log S - T / S,
// and gathers the given labels.  A row of a single chunk needs one kernel.
// Everything is fp32 in a fixed order; logits are only compared and
// subtracted before the exponential (z - M is exact or rounded once).
#include "elem.h"

namespace haste {

namespace {

constexpr int NT = 256;
constexpr float kNegInf = -__builtin_inff();

// A candidate's key: larger is better (value descending, then label
// ascending); 0: none.
typedef unsigned long long key_t;
__device__ __forceinline__ key_t cand_key(float v, unsigned label) {
    return ((key_t)f32_order_key(v) << 32) | (0xffffffffu - label);
}
__device__ __forceinline__ bool is_cand(float v) { return v > kNegInf; }   // false for NaN

// S = 0: no logit above -inf (M = -inf).  A NaN or +inf ends as NaN in S.
struct Stat {
    float m, S, T;
};
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
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    Stat r = s[0];
    for (int i = 1; i < NT / 64; ++i) r = stat_join(r, s[i]);
    return r;
}
__device__ __forceinline__ key_t block_max(key_t k, key_t *s) {
    for (int o = 32; o > 0; o >>= 1) {
        const key_t t = __shfl_xor(k, o, 64);
        k = t > k ? t : k;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = k;
    __syncthreads();
    for (int i = 0; i < NT / 64; ++i) k = s[i] > k ? s[i] : k;
    return k;
}

// How rows are cut: vectors of 16 bytes, aligned in memory (a row that starts
// inside one shares it with what is before).
struct Cut {
    int nc[2];        // chunks of the parts
    int per[2];       // vectors a chunk
    int nv;           // vectors a thread, at most
    int64_t items;    // B * (nc[0] + nc[1])
    __host__ __device__ int chunks() const { return nc[0] + nc[1]; }
};

Cut cut_rows(int B, int64_t H, int64_t L, bool bf) {
    const int V = bf ? 8 : 4;
    const int64_t n[2] = {H, L};
    int64_t vec[2];
    for (int p = 0; p < 2; ++p) vec[p] = n[p] ? (n[p] + 2 * V - 2) / V : 0;   // from any start
    Cut c{};
    auto set = [&](int nv) {
        c.nv = nv;
        for (int p = 0; p < 2; ++p) {
            c.nc[p] = (int)((vec[p] + NT * nv - 1) / (NT * nv));
            c.per[p] = c.nc[p] ? (int)((vec[p] + c.nc[p] - 1) / c.nc[p]) : 0;
        }
        c.items = (int64_t)B * c.chunks();
    };
    // A single chunk (one launch) where it can be; else the largest chunks
    // that still give every CU a few workgroups.
    const bool one = (H == 0 || L == 0) && vec[0] + vec[1] <= 16 * NT;
    int nv = one ? 2 : 16;
    set(nv);
    if (one)
        while (c.chunks() > 1) set(nv *= 2);
    else
        while (nv > 2 && c.items < 1024) set(nv /= 2);
    return c;
}

// workspace: keys (B x chunks x K), stats (B x chunks), row losses (B)
struct Ws {
    Stat *stat;
    key_t *key;
    float *loss;
};
__host__ __device__ inline Ws ws_map(const LogprobArgs &a, int64_t items) {
    Ws w;
    w.key = (key_t *)a.ws;
    w.stat = (Stat *)(w.key + items * a.K);
    w.loss = (float *)(w.stat + items);
    return w;
}

constexpr int CAP = 512;      // candidates that are ranked in LDS
struct Shared {
    Stat st[NT / 64];
    key_t key[NT / 64];
    float f[NT / 64], g[NT / 64];
    int n;
    key_t list[CAP];
    key_t top[8];
};

// The K best of the n <= CAP keys in sh.list, in order, into sh.top (0 where
// there are fewer).  All keys differ, so their ranks do.
__device__ __forceinline__ void rank_keys(Shared &sh, int n, int K) {
    if ((int)threadIdx.x < K && (int)threadIdx.x >= n) sh.top[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < n; i += NT) {
        const key_t k = sh.list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.list[j] > k ? 1 : 0;
        if (rank < K) sh.top[rank] = k;
    }
    __syncthreads();
}

// A value that at least eight of the workgroup's 256 values reach (K <= 8):
// the smallest of the eight maxima of a wave's lane octets, the best of the
// waves'.  Below it nothing belongs to the K best.
__device__ __forceinline__ float threshold8(float v, Shared &sh) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
#pragma unroll
    for (int o = 8; o < 64; o <<= 1) v = fminf(v, __shfl_xor(v, o, 64));
    if ((threadIdx.x & 63) == 0) sh.g[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(sh.g[0], sh.g[1]), fmaxf(sh.g[2], sh.g[3]));
}

// A row's results from its statistics and, in sh.top, its K best keys.
template <bool BF>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, int64_t b, const Stat &st, Shared &sh, float *row_loss) {
    const bool none = st.S == 0.f;
    const float logS = none ? 0.f : logf(st.S);
    const float lse = none ? kNegInf : st.m + logS;
    if (threadIdx.x == 0) {
        a.lse[b] = lse;
        if (a.entropy) a.entropy[b] = none ? 0.f : logS - st.T / st.S;
    }
    if ((int)threadIdx.x < a.K) {
        const key_t k = sh.top[threadIdx.x];
        a.top_v[b * a.K + threadIdx.x] = k ? f32_from_order_key((unsigned)(k >> 32)) - lse : kNegInf;
        a.top_i[b * a.K + threadIdx.x] = k ? (int32_t)(a.off + (0xffffffffu - (unsigned)k)) : -1;
    }
    if (!a.row_ptr || (!a.logp && !a.loss)) return;
    const int e0 = max(a.row_ptr[b], 0), e1 = min(a.row_ptr[b + 1], a.nnz);
    float sum = 0.f;
    for (int e = e0 + threadIdx.x; e < e1; e += NT) {
        const int64_t j = (int64_t)a.labels[e] - a.off;
        float lp = kNegInf;
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
    if ((threadIdx.x & 63) == 0) sh.f[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) row_loss[b] = sh.f[0] + sh.f[1] + sh.f[2] + sh.f[3];
}

// element j of a 16-byte vector
template <bool BF>
__device__ __forceinline__ float elem(const u32x4 &r, int j) {
    if (BF) return __uint_as_float(j & 1 ? r[j >> 1] & 0xffff0000u : r[j >> 1] << 16);
    return __uint_as_float(r[j]);
}

// The same registers, taken for new values: each pass over them unpacks its
// logits again (one instruction each) instead of keeping 128 floats alive.
template <int NV>
__device__ __forceinline__ void renew(u32x4 (&r)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(r[k][j]));
}

// vector v of a row of n elements at p; the row starts `shift` elements into
// vector 0 (p16); elements outside the row read as -inf
template <bool BF>
__device__ __forceinline__ u32x4 load_vec(const u32x4 *p16, int64_t v, int shift, int64_t n) {
    constexpr int V = BF ? 8 : 4;
    const int64_t e = v * V - shift;
    if (e >= 0 && e + V <= n) return p16[v];
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = BF ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (e + j < 0 || e + j >= n) continue;
        if (BF) {
            const unsigned t = ((const unsigned short *)(p16 + v))[j];
            r[j >> 1] = j & 1 ? (r[j >> 1] & 0xffffu) | t << 16 : (r[j >> 1] & 0xffff0000u) | t;
        } else {
            r[j] = ((const unsigned *)(p16 + v))[j];
        }
    }
    return r;
}

}  // namespace

size_t logprob_ws_bytes(int B, int64_t H, int64_t L, bool bf, int K) {
    const int64_t items = cut_rows(B, H, L, bf).items;
    return (size_t)items * K * 8 + (size_t)items * sizeof(Stat) + (size_t)B * 4;
}

// One chunk a workgroup, in registers: NV vectors a thread.  Bound by the
// reading: per bf16 logit twelve issue slots (the exponential is four), less
// than the 2 bytes take to arrive.
template <bool BF, int NV, bool ONE>
__global__ __launch_bounds__(NT) void k_lp_stats(LogprobArgs a, Cut cut) {
    constexpr int V = BF ? 8 : 4;
    __shared__ Shared sh;
    const unsigned tid = threadIdx.x, nc = (unsigned)cut.chunks();
    const Ws w = ws_map(a, cut.items);
    for (unsigned item = blockIdx.x; item < (unsigned)cut.items; item += gridDim.x) {
        const unsigned b = ONE ? item : item / nc, c = ONE ? 0 : item - b * nc;
        const int p = c >= (unsigned)cut.nc[0];
        const int64_t n = a.n[p];
        const int64_t v0 = (int64_t)(p ? c - cut.nc[0] : c) * cut.per[p];
        const uintptr_t row = (uintptr_t)a.z[p] + (uintptr_t)((int64_t)b * a.ld[p]) * (BF ? 2 : 4);
        const u32x4 *p16 = (const u32x4 *)(row & ~(uintptr_t)15);
        const int shift = (int)(row & 15) / (BF ? 2 : 4);

        u32x4 raw[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * NT + (int)tid;
            if (i < cut.per[p]) raw[k] = load_vec<BF>(p16, v0 + i, shift, n);
            else
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[k][j] = BF ? 0xff80ff80u : 0xff800000u;
        }
        float top[NV], mine = kNegInf;      // the vectors' and the thread's largest logits
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            top[k] = kNegInf;
#pragma unroll
            for (int j = 0; j < V; ++j) top[k] = fmaxf(top[k], elem<BF>(raw[k], j));
            mine = fmaxf(mine, top[k]);
        }
        float M = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) M = fmaxf(M, __shfl_xor(M, o, 64));
        if ((tid & 63) == 0) sh.f[tid >> 6] = M;
        if (tid == 0) sh.n = 0;
        __syncthreads();
        M = fmaxf(fmaxf(sh.f[0], sh.f[1]), fmaxf(sh.f[2], sh.f[3]));
        renew(raw);
        const float M0 = M == kNegInf ? 0.f : M;
        float S = 0.f, T = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = elem<BF>(raw[k], j) - M0;
                const float e = __builtin_amdgcn_exp2f(v * kLog2e);
                S += e;
                T = __builtin_fmaf(e, fmaxf(v, -1e4f), T);   // a masked logit: 0 * -1e4, not 0 * -inf
            }
        S = wave_sum(S);
        T = wave_sum(T);
        Stat st;
        if ((tid & 63) == 0) sh.st[tid >> 6] = (Stat){M, S, T};
        const unsigned l0 = (unsigned)((p ? a.n[0] : 0) + v0 * V - shift);   // label of the chunk's first element
        if (a.K > 0) {
            const float tau = threshold8(mine, sh);      // its barrier also publishes sh.st
            unsigned hit = 0;                            // vectors that reach it
#pragma unroll
            for (int k = 0; k < NV; ++k) hit |= (top[k] >= tau ? 1u : 0u) << k;
            while (hit) {                                // read again (a few of the chunk's 32 K logits)
                const int k = __ffs(hit) - 1;
                hit &= hit - 1;
                const u32x4 r = load_vec<BF>(p16, v0 + k * NT + tid, shift, n);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float z = elem<BF>(r, j);
                    if (!(z >= tau) || !is_cand(z)) continue;
                    const int at = atomicAdd(&sh.n, 1);
                    if (at < CAP) sh.list[at] = cand_key(z, l0 + (unsigned)(k * NT + (int)tid) * V + j);
                }
            }
            __syncthreads();
            if (sh.n <= CAP && tau == tau) {
                rank_keys(sh, sh.n, a.K);
            } else {
                // Very many equal logits (or a signalling NaN, which no
                // comparison passes): the best one below the last, K times.
                key_t last = ~(key_t)0;
                for (int q = 0; q < a.K; ++q) {
                    key_t best = 0;
#pragma unroll 1
                    for (int i = tid; i < cut.per[p]; i += NT) {
                        const u32x4 r = load_vec<BF>(p16, v0 + i, shift, n);
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float z = elem<BF>(r, j);
                            const key_t key = is_cand(z) ? cand_key(z, l0 + (unsigned)i * V + j) : 0;
                            if (key < last && key > best) best = key;
                        }
                    }
                    last = block_max(best, sh.key);
                    if (tid == 0) sh.top[q] = last;
                }
                __syncthreads();
            }
        } else {
            __syncthreads();
        }
        st.m = M;
        st.S = sh.st[0].S + sh.st[1].S + sh.st[2].S + sh.st[3].S;
        st.T = sh.st[0].T + sh.st[1].T + sh.st[2].T + sh.st[3].T;
        if (ONE) {
            finish_row<BF>(a, b, st, sh, w.loss);
        } else {
            if (tid == 0) w.stat[item] = st;
            if ((int)tid < a.K) w.key[(int64_t)item * a.K + tid] = sh.top[tid];
        }
        __syncthreads();      // the next item's use of sh
    }
}

// A row's chunks joined, one workgroup a row.
template <bool BF>
__global__ __launch_bounds__(NT) void k_lp_rows(LogprobArgs a, Cut cut) {
    __shared__ Shared sh;
    const int nc = cut.chunks();
    const Ws w = ws_map(a, cut.items);
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (threadIdx.x == 0) sh.n = 0;
        Stat st = {kNegInf, 0.f, 0.f};
        for (int c = threadIdx.x; c < nc; c += NT) st = stat_join(st, w.stat[b * nc + c]);
        st = block_join(st, sh.st);
        if (a.K > 0) {
            const key_t *key = w.key + b * nc * a.K;
            const int n = nc * a.K;
            key_t best = 0;
            for (int i = threadIdx.x; i < n; i += NT) best = key[i] > best ? key[i] : best;
            // a key that eight of the 256 threads' best reach (as threshold8)
            key_t t = best;
            for (int o = 1; o < 8; o <<= 1) {
                const key_t x = __shfl_xor(t, o, 64);
                t = x > t ? x : t;
            }
            for (int o = 8; o < 64; o <<= 1) {
                const key_t x = __shfl_xor(t, o, 64);
                t = x < t ? x : t;
            }
            if ((threadIdx.x & 63) == 0) sh.key[threadIdx.x >> 6] = t;
            __syncthreads();
            for (int i = 0; i < NT / 64; ++i) t = sh.key[i] > t ? sh.key[i] : t;
            if (best >= t)
                for (int i = threadIdx.x; i < n; i += NT) {
                    const key_t k = key[i];
                    if (k < t || k == 0) continue;
                    const int at = atomicAdd(&sh.n, 1);
                    if (at < CAP) sh.list[at] = k;
                }
            __syncthreads();
            if (sh.n <= CAP) {
                rank_keys(sh, sh.n, a.K);
            } else {
                key_t last = ~(key_t)0;
                for (int q = 0; q < a.K; ++q) {
                    best = 0;
                    for (int i = threadIdx.x; i < n; i += NT)
                        if (key[i] < last && key[i] > best) best = key[i];
                    last = block_max(best, sh.key);
                    if (threadIdx.x == 0) sh.top[q] = last;
                }
                __syncthreads();
            }
        }
        finish_row<BF>(a, b, st, sh, w.loss);
        __syncthreads();
    }
}

// *loss += s * the sum of the rows' losses, in a fixed order
__global__ __launch_bounds__(NT) void k_lp_loss(LogprobArgs a, Cut cut) {
    __shared__ float sl[NT / 64];
    const Ws w = ws_map(a, cut.items);
    float t = 0.f;
    for (int b = threadIdx.x; b < a.B; b += NT) t += w.loss[b];
    t = wave_sum(t);
    if ((threadIdx.x & 63) == 0) sl[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) *a.loss += a.s * (sl[0] + sl[1] + sl[2] + sl[3]);
}

template <bool BF>
static hipError_t launch_fwd(const LogprobArgs &a, hipStream_t st) {
    const Cut cut = cut_rows(a.B, a.n[0], a.n[1], a.bf);
    const unsigned most = 1u << 22;
    const dim3 grid((unsigned)(cut.items < most ? cut.items : most)), rows((unsigned)(a.B < (1 << 22) ? a.B : 1 << 22));
#define GO(NV, ONE) hipLaunchKernelGGL((k_lp_stats<BF, NV, ONE>), grid, dim3(NT), 0, st, a, cut)
    if (cut.chunks() == 1) {
        if (cut.nv == 2) GO(2, true);
        else if (cut.nv == 4) GO(4, true);
        else if (cut.nv == 8) GO(8, true);
        else GO(16, true);
    } else {
        if (cut.nv == 2) GO(2, false);
        else if (cut.nv == 4) GO(4, false);
        else if (cut.nv == 8) GO(8, false);
        else GO(16, false);
        hipLaunchKernelGGL(k_lp_rows<BF>, rows, dim3(NT), 0, st, a, cut);
    }
#undef GO
    if (a.loss) hipLaunchKernelGGL(k_lp_loss, dim3(1), dim3(NT), 0, st, a, cut);
    return hipGetLastError();
}

bool logprob_supported(int B, int64_t H, int64_t L, bool bf) { return cut_rows(B, H, L, bf).items <= INT32_MAX; }

hipError_t launch_logprob_fwd(const LogprobArgs &a, hipStream_t st) {
    return a.bf ? launch_fwd<true>(a, st) : launch_fwd<false>(a, st);
}

// --------------------------------------------------------------- backward
namespace {

// dz of one logit, before its labels' own gradients: -p (G + n (log p + H));
// a masked logit has p = 0 and log p = -inf, kept finite by the clamp
template <bool ENT>
__device__ __forceinline__ float dz_dense(float z, float lse, float G, float n, float H) {
    const float lp = z - lse, p = __builtin_amdgcn_exp2f(lp * kLog2e);
    return ENT ? -p * (G + n * (fmaxf(lp, -1e4f) + H)) : -p * G;
}

constexpr int BV = 8;      // vectors a thread

}  // namespace

// A chunk of 2048 vectors a workgroup, vectors aligned in dz.  Reads every
// logit once and writes its gradient once; the given labels' own gradients
// are added by rewriting their elements after the barrier.
template <bool BF, bool ENT>
__global__ __launch_bounds__(NT) void k_lp_bwd(LogprobArgs a, int nc0, int nc, int64_t items) {
    constexpr int V = BF ? 8 : 4, ES = BF ? 2 : 4;
    __shared__ float sg[NT / 64];
    const int tid = threadIdx.x;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const unsigned b = (unsigned)item / (unsigned)nc, c = (unsigned)item - b * (unsigned)nc;
        const int p = c >= (unsigned)nc0;
        const int64_t n = a.n[p], v0 = (int64_t)(p ? c - nc0 : c) * (NT * BV);
        const char *zr = (const char *)a.z[p] + (int64_t)b * a.ld[p] * ES;
        char *dr = (char *)a.dz[p] + (int64_t)b * n * ES;
        const int shift = (int)((uintptr_t)dr & 15) / ES;
        u32x4 raw[BV];
#pragma unroll
        for (int k = 0; k < BV; ++k) {
            const int64_t e = (v0 + k * NT + tid) * V - shift;
            if (e >= 0 && e + V <= n) {
                if (BF) raw[k] = *(const u32x4h *)(zr + e * ES);
                else raw[k] = *(const u32x4w *)(zr + e * ES);
            }
        }
        const float lse = a.lse[b];
        const bool none = lse == kNegInf;
        const float nn = ENT ? a.dent[b] : 0.f, H = ENT ? a.entropy[b] : 0.f;
        int e0 = 0, e1 = 0;
        if (a.row_ptr) {
            e0 = max(a.row_ptr[b], 0);
            e1 = min(a.row_ptr[b + 1], a.nnz);
        }
        const int64_t N = a.n[0] + a.n[1];
        float G = 0.f;
        if (e1 - e0 <= 8) {      // the same for every thread
            for (int e = e0; e < e1; ++e) {
                const int64_t j = (int64_t)a.labels[e] - a.off;
                if (j >= 0 && j < N) G += a.dlogp ? a.dlogp[e] : -a.s;
            }
        } else {
            for (int e = e0 + tid; e < e1; e += NT) {
                const int64_t j = (int64_t)a.labels[e] - a.off;
                if (j >= 0 && j < N) G += a.dlogp ? a.dlogp[e] : -a.s;
            }
            G = wave_sum(G);
            if ((tid & 63) == 0) sg[tid >> 6] = G;
            __syncthreads();
            G = sg[0] + sg[1] + sg[2] + sg[3];
        }
#pragma unroll
        for (int k = 0; k < BV; ++k) {
            const int64_t e = (v0 + k * NT + tid) * V - shift;
            if (e >= 0 && e + V <= n) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = none ? 0.f : dz_dense<ENT>(elem<BF>(raw[k], j), lse, G, nn, H);
                u32x4 r;
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = BF ? pack_bf16x2(o[2 * j % V], o[(2 * j + 1) % V]) : __float_as_uint(o[j % V]);
                *(u32x4 *)(dr + e * ES) = r;
            } else if (e < n) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (e + j >= 0 && e + j < n)
                        store1<BF>(dr, e + j, none ? 0.f : dz_dense<ENT>(load1<BF>(zr, e + j), lse, G, nn, H));
            }
        }
        if (none || e1 <= e0) continue;      // uniform
        // the chunk's given labels, each by the thread of its first entry
        __syncthreads();
        const int64_t first = v0 * V - shift, l0 = (p ? a.n[0] : 0);
        for (int e = e0 + tid; e < e1; e += NT) {
            const int32_t id = a.labels[e];
            const int64_t j = (int64_t)id - a.off - l0;      // element of the part's row
            if (j < 0 || j >= n || j < first || j >= first + (int64_t)NT * BV * V) continue;
            float g = 0.f;
            bool mine = true;
            for (int f = e0; f < e1; ++f) {
                if (a.labels[f] != id) continue;
                if (f < e) mine = false;
                g += a.dlogp ? a.dlogp[f] : -a.s;
            }
            if (mine) store1<BF>(dr, j, g + dz_dense<ENT>(load1<BF>(zr, j), lse, G, nn, H));
        }
    }
}

hipError_t launch_logprob_bwd(const LogprobArgs &a, hipStream_t st) {
    const int V = a.bf ? 8 : 4;
    int64_t nc[2];
    for (int p = 0; p < 2; ++p) nc[p] = a.n[p] ? ((a.n[p] + 2 * V - 2) / V + NT * BV - 1) / (NT * BV) : 0;
    const int64_t items = (nc[0] + nc[1]) * a.B;
    if (items > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(items < (1 << 22) ? items : 1 << 22));
#define GO(BF, ENT) \
    hipLaunchKernelGGL((k_lp_bwd<BF, ENT>), grid, dim3(NT), 0, st, a, (int)nc[0], (int)(nc[0] + nc[1]), items)
    if (a.bf && a.dent) GO(true, true);
    else if (a.bf) GO(true, false);
    else if (a.dent) GO(false, true);
    else GO(false, false);
#undef GO
    return hipGetLastError();
}

}  // namespace haste
