// logprob.hip -- softmax statistics over head and tail logits: log
// probabilities of given labels, entropy, top alternatives, and the gradient.
//
// One reading of the logits.  A row's head and tail parts are cut into chunks
// of at most 128 KB (lp_cut.h).  A workgroup goes over its chunk, of which up to
// 64 KB stay in registers, and forms
//   M = max z, S = sum e^(z - M), T = sum e^(z - M) (z - M)
// and the chunk's K best logits; a second kernel joins a row's chunks,
//   S = sum_c S_c e^(M_c - M),  T = sum_c e^(M_c - M) (T_c + (M_c - M) S_c),
//   lse = M + log S,  entropy = log S - T / S,
// and gathers the given labels.  A row of a single chunk needs one kernel.
// Everything is fp32 in an order that the row's place in memory fixes; before
// the exponential a logit is compared and once rounded (k_lp_stats).
//
// Bound by memory at training sizes: 512 rows of 670,192 bf16 logits 121.5 us and
// 7.3 for the join, 5.5 TB/s (a copy of 1 GiB: 5.2); the gradient 250 us, 5.5 TB/s.
// A single row of 8.6M: 9 us and 5, of which the 17 MB are 3.3: two launches and
// the latency of picking the best labels (without them 6.2 and 2.7).
#include "elem.h"
#include "lp_cut.h"

namespace haste {

namespace {

constexpr int NT = kLpThreads;
constexpr float kNegInf = -__builtin_inff();

// A candidate's key: larger is better (value descending, then label
// ascending); 0: none.
typedef unsigned long long key_t;
__device__ __forceinline__ key_t cand_key(float v, unsigned label) {
    return ((key_t)f32_order_key(v) << 32) | (0xffffffffu - label);
}
__device__ __forceinline__ bool is_cand(float v) { return v > kNegInf; }   // false for NaN
__device__ __forceinline__ bool pass(float v, float tau) { return v >= tau && v > kNegInf; }

// S = 0: no logit above -inf (M = -inf).  A NaN or +inf ends as NaN in S.
struct Stat {
    float m, S, T;
};
// n statistics joined
template <int N>
__device__ __forceinline__ Stat stat_join(const Stat (&q)[N]) {
    Stat r = {kNegInf, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) r.m = fmaxf(r.m, q[i].m);
    const float m0 = r.m == kNegInf ? 0.f : r.m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = q[i].m - m0, f = __expf(d);      // d = -inf, f = 0 for an empty one
        r.S += f * q[i].S;
        r.T += f * (q[i].T + fmaxf(d, -1e4f) * q[i].S);
    }
    return r;
}
// over the workgroup; s: room for one a wave
__device__ __forceinline__ Stat block_join(Stat v, Stat *s) {
    const float M = f32_from_order_key(wave_max_dpp(f32_order_key(v.m)));
    const float d = v.m - (M == kNegInf ? 0.f : M), f = __expf(d);
    const float S = wave_sum_dpp(f * v.S), T = wave_sum_dpp(f * (v.T + fmaxf(d, -1e4f) * v.S));
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = (Stat){M, S, T};
    __syncthreads();
    const Stat q[NT / 64] = {s[0], s[1], s[2], s[3]};
    return stat_join(q);
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

constexpr int BAT = kLpBatch;

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
constexpr int SLOTS = 64;     // batches that are searched at a time
struct Shared {
    Stat st[NT / 64];
    key_t key[NT / 64];
    float f[NT / 64];
    unsigned u[NT / 64];
    unsigned best[NT];
    int n, slots;
    key_t list[CAP];
    key_t top[8];
    __attribute__((aligned(16))) u32x4 batch[SLOTS][BAT];
    unsigned from[SLOTS];
};

// The K-th largest (K <= 8) of the largest values of 16 groups of the workgroup's
// threads: K of the values reach it, few more do.  Thread t is in group t % 16, so
// that a run of neighbouring logits is spread over the groups.  kth_put before a
// barrier, kth_get after it.
__device__ __forceinline__ void kth_put(unsigned v, Shared &sh) { sh.best[threadIdx.x] = v; }
template <int I>
__device__ __forceinline__ void kth_count(unsigned v, int &above, int &reach) {
    const unsigned t = dpp_u32<0x120 + I>(v);      // the row's lanes rotated by I
    above += t > v ? 1 : 0;
    reach += t >= v ? 1 : 0;
    if constexpr (I < 15) kth_count<I + 1>(v, above, reach);
}
__device__ __forceinline__ unsigned kth_get(int K, const Shared &sh) {
    unsigned v = 0;
#pragma unroll
    for (int i = 0; i < NT / 16; ++i) v = max(v, sh.best[16 * i + (threadIdx.x & 15)]);
    int above = 0, reach = 1;
    kth_count<1>(v, above, reach);
    return lane_u32(v, __ffsll((unsigned long long)__ballot(above < K && reach >= K)) - 1);
}
// The K best of the n <= CAP keys in sh.list, in order, into sh.top (0 where
// there are fewer).  All keys differ, so their ranks do.  A lane a key while a
// wave has room for them (nearly always): no reading from LDS between.
__device__ __forceinline__ void rank_keys(Shared &sh, int n, int K) {
    n = __builtin_amdgcn_readfirstlane(n);
    if ((int)threadIdx.x < K && (int)threadIdx.x >= n) sh.top[threadIdx.x] = 0;
    if (n <= 64) {
        if (threadIdx.x < 64) {
            const key_t k = (int)threadIdx.x < n ? sh.list[threadIdx.x] : 0;
            int rank = 0;
#pragma unroll 1
            for (int j = 0; j < n; ++j)
                rank += ((key_t)lane_u32((unsigned)(k >> 32), j) << 32 | lane_u32((unsigned)k, j)) > k ? 1 : 0;
            if (k && rank < K) sh.top[rank] = k;
        }
    } else {
        for (int i = threadIdx.x; i < n; i += NT) {
            const key_t k = sh.list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += sh.list[j] > k ? 1 : 0;
            if (rank < K) sh.top[rank] = k;
        }
    }
    __syncthreads();
}

// The given labels of a row, and the thread's first one's logit, read ahead.
struct Given {
    int e0, e1;
    float z;         // -inf: outside the range (or none)
    bool in;
};
template <bool BF>
__device__ __forceinline__ float given_logit(const LogprobArgs &a, int64_t b, int e, bool *in) {
    const int64_t j = (int64_t)a.labels[e] - a.off;
    *in = j >= 0 && j < a.n[0] + a.n[1];
    if (!*in) return kNegInf;
    const int p = j >= a.n[0];
    return load1<BF>(a.z[p], b * a.ld[p] + (p ? j - a.n[0] : j));
}
template <bool BF>
__device__ __forceinline__ Given read_given(const LogprobArgs &a, int64_t b) {
    Given g = {0, 0, kNegInf, false};
    if (!a.row_ptr || (!a.logp && !a.loss)) return g;
    g.e0 = max(a.row_ptr[b], 0);
    g.e1 = min(a.row_ptr[b + 1], a.nnz);
    if (g.e0 + (int)threadIdx.x < g.e1) g.z = given_logit<BF>(a, b, g.e0 + threadIdx.x, &g.in);
    return g;
}

// A row's results from its statistics and, in sh.top, its K best keys.
template <bool BF>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, int64_t b, const Stat &st, const Given &given, Shared &sh,
                                           float *row_loss) {
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
    float sum = 0.f;
    for (int e = given.e0 + threadIdx.x; e < given.e1; e += NT) {
        float z = given.z;
        bool in = given.in;
        if (e >= given.e0 + NT) z = given_logit<BF>(a, b, e, &in);
        const float lp = none || !in ? kNegInf : z - lse;
        if (in) sum -= lp;
        if (a.logp) a.logp[e] = lp;
    }
    if (!a.loss) return;
    sum = wave_sum_dpp(sum);
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

// A chunk of a row: cnt whole vectors from p (aligned), element e0 of the row
// the first of them, and single elements before and after them where the row
// starts or ends inside a vector (fewer than a vector each), one a thread.
template <bool BF>
struct Chunk {
    static constexpr int V = BF ? 8 : 4;
    const u32x4 *p;
    int64_t e0;
    int cnt;
    int64_t single;      // the thread's own single element, or -1
    // chunk c of `per` vectors of a row of n elements at row
    __device__ __forceinline__ Chunk(const char *row, int64_t n, int64_t c, int per) {
        const int over = (int)((uintptr_t)row & 15), shift = over / (16 / V);
        const int64_t first = c * per * V - shift;                    // element 0 of the chunk's vectors
        const int lo = first < 0 ? 1 : 0;
        const int64_t left = n - first;                               // below V: nothing whole
        const int hi = left <= 0 ? 0 : (int)min((int64_t)per, left / V);
        p = (const u32x4 *)(row - over) + c * per + lo;
        e0 = first + lo * V;
        cnt = max(0, hi - lo);
        const int t = (int)threadIdx.x;
        const int64_t tail = first + (int64_t)hi * V;                 // first element after the whole vectors
        single = -1;
        if (first < 0 && t < V && t < V - shift && t < n) single = t;
        else if (hi < per && tail >= 0 && t >= V && t < 2 * V && tail + t - V < n) single = tail + t - V;
    }
};

}  // namespace

size_t logprob_ws_bytes(int B, int64_t H, int64_t L, bool bf, int K) {
    const int64_t items = cut_rows(B, H, L, bf).items;
    return (size_t)items * K * 8 + (size_t)items * sizeof(Stat) + (size_t)B * 4;
}

// One chunk a workgroup, NB batches of four vectors a thread.  Up to four
// batches are loaded at once and stay in registers until the best are picked
// from them; of eight, the next one's loads are under way while one is summed,
// and the few batches that hold one of the best are read again.
//
// The sums run in the exponent's own base and relative to the thread's own
// largest logit m so far: with c = m log2(e) rounded, u = fma(z, log2(e), -c) is
// one rounding, S' = sum 2^u, T' = sum 2^u u.  When m grows, S' and T' move to the
// new c; what the rounding of the last c shifted every u by, r = fma(m, log2(e),
// -c), is exact and taken out at the end: S = 2^-r S', T = 2^-r (T' - r S') / log2(e).
// c comes from max(m, -1e6), so that masked logits alone leave S' = 0.  That S' is
// not relative to an m below -1e6, which shows no more where the chunk's largest
// logit is 128 above (e^-128 of it).  Chunks whose largest logit is below that, or
// at 1e6 and above (r would no longer be small), are summed again without c.
//
// Per bf16 logit: unpack, half a maximum, fma, exponential, add, clamp, fma: at
// 5.5 TB/s about as long as the memory takes, which is why the sums run in the
// exponent's base (with a natural exponential and a shared maximum 202 us, the
// form here 121).
template <bool BF, int NB, bool ONE>
__global__ __launch_bounds__(NT) void k_lp_stats(LogprobArgs a, Cut cut) {
    constexpr int V = BF ? 8 : 4, ES = BF ? 2 : 4, NE = BAT * V;
    constexpr bool KEEP = NB <= 4;
    constexpr float kBig = 1e6f, kLow = 128.f - kBig;
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const unsigned nc = (unsigned)cut.chunks();
    const Ws w = ws_map(a, cut.items);
    for (unsigned item = blockIdx.x; item < (unsigned)cut.items; item += gridDim.x) {
        const unsigned b = ONE ? item : item / nc, c = ONE ? 0 : item - b * nc;
        const int p = c >= (unsigned)cut.nc[0];
        const char *row = (const char *)a.z[p] + (int64_t)b * a.ld[p] * ES;
        const Chunk<BF> ch(row, a.n[p], p ? c - cut.nc[0] : c, cut.per[p]);
        // batch i, its vectors past the end for the last one (nothing whole at
        // all: not read); mask() then makes those -inf
        const int last_v = ch.cnt - 1;
        auto load = [&](int i, u32x4 (&r)[BAT]) {
#pragma unroll
            for (int k = 0; k < BAT; ++k)
                r[k] = *(const u32x4 *)((const char *)ch.p + 16u * (unsigned)min((i * BAT + k) * NT + tid, last_v));
        };
        auto mask = [&](int i, u32x4 (&r)[BAT]) {
            if ((i + 1) * BAT * NT <= ch.cnt) return;       // uniform
            const unsigned x = BF ? 0xff80ff80u : 0xff800000u;
#pragma unroll
            for (int k = 0; k < BAT; ++k)
                if ((i * BAT + k) * NT + tid > last_v) r[k] = (u32x4){x, x, x, x};
        };
        u32x4 raw[KEEP ? NB : 2][BAT];
#pragma unroll
        for (int i = 0; i < (KEEP ? NB : 1); ++i)
            if (i * BAT * NT <= last_v) load(i, raw[i]);
        const float zs = ch.single >= 0 ? load1<BF>(row, ch.single) : kNegInf;
        Given given{};
        if (ONE) given = read_given<BF>(a, b);
        float top[NB], m = kNegInf, cm = -kBig * kLog2e, S = 0.f, T = 0.f;
        auto move_to = [&](float x) {       // m = max(m, x)
#pragma clang fp contract(off)              // d is the step of the rounded c, not of the product
            m = fmaxf(m, x);
            const float cn = fmaxf(m, -kBig) * kLog2e, d = cm - cn, f = __builtin_amdgcn_exp2f(d);
            T = f * __builtin_fmaf(d, S, T);
            S *= f;
            cm = cn;
        };
        auto add = [&](float z) {
            const float u = __builtin_fmaf(z, kLog2e, -cm);
            const float e = __builtin_amdgcn_exp2f(u);
            S += e;
            T = __builtin_fmaf(e, fmaxf(u, -1e4f), T);      // a masked logit: 0 * -1e4, not 0 * -inf
        };
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            top[i] = kNegInf;
            if (i * BAT * NT >= ch.cnt) continue;           // uniform: nothing (more)
            if (!KEEP && i + 1 < NB) load(i + 1, raw[(i + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);      // one batch ahead, no more: registers
            u32x4 (&now)[BAT] = raw[KEEP ? i : i & 1];
            mask(i, now);
            float z[NE];
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                z[j] = elem<BF>(now[j / V], j % V);
                top[i] = fmaxf(top[i], z[j]);
            }
            move_to(top[i]);
#pragma unroll
            for (int j = 0; j < NE; ++j) add(z[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        move_to(zs);
        add(zs);
        Stat st = {m, S, T};
        {
            const float r = __builtin_fmaf(fmaxf(m, -kBig), kLog2e, -cm), f = __builtin_amdgcn_exp2f(-r);
            st.S = f * S;
            st.T = f * (T - r * S) * kLn2;
        }
        // tau: a value that K of the logits reach; below it nothing belongs to the K best
        kth_put(f32_order_key(m), sh);
        if (tid == 0) sh.n = sh.slots = 0;
        st = block_join(st, sh.st);       // its barrier publishes sh.best too
        float tau = a.K > 0 ? f32_from_order_key(kth_get(a.K, sh)) : 0.f;
        if ((st.m >= kBig || st.m < kLow) && st.m != kNegInf) {
            const float M = st.m, vs = zs - M;
            S = __builtin_amdgcn_exp2f(vs * kLog2e);
            T = S * fmaxf(vs, -1e4f);
#pragma unroll 1
            for (int i = tid; i < ch.cnt; i += NT) {
                const u32x4 q = ch.p[i];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float v = elem<BF>(q, j) - M;
                    const float e = __builtin_amdgcn_exp2f(v * kLog2e);
                    S += e;
                    T = __builtin_fmaf(e, fmaxf(v, -1e4f), T);
                }
            }
            __syncthreads();              // sh.st has been read
            st = block_join((Stat){M, S, T}, sh.st);
        }
        const unsigned lp = (unsigned)(p ? a.n[0] : 0), l0 = lp + (unsigned)ch.e0;   // labels of the part's and the vectors' first element
        if (a.K > 0 && st.S != st.S) {
            // A NaN (or an infinity) among them, the same for all threads.  A
            // signalling one upsets the maxima: the hardware's maximum returns
            // it, quieted.  Once more by comparisons, which no NaN passes, a
            // thread's largest logit for all of its batches.
            m = is_cand(zs) ? zs : kNegInf;
#pragma unroll 1
            for (int i = tid; i < ch.cnt; i += NT) {
                const u32x4 q = ch.p[i];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float z = elem<BF>(q, j);
                    m = z > m ? z : m;
                }
            }
#pragma unroll
            for (int i = 0; i < NB; ++i)
                if (i * BAT * NT < ch.cnt) top[i] = m;      // others have no data
            __syncthreads();              // sh.best has been read
            kth_put(f32_order_key(m), sh);
            __syncthreads();
            tau = f32_from_order_key(kth_get(a.K, sh));
        }
        if (a.K > 0) {
            // The logits above tau, or (ties) reaching it, into sh.list.  The few
            // batches that hold any pass through LDS, where the whole workgroup
            // searches them: short code, since a small call runs it once and waits
            // for every line of it.
            auto gather = [&](bool ties) {
                auto take = [&](float z) { return (ties ? z >= tau : z > tau) && is_cand(z); };
                unsigned hit = 0;                        // the thread's batches that have any
#pragma unroll
                for (int i = 0; i < NB; ++i) hit |= (take(top[i]) ? 1u : 0u) << i;
                if (pass(zs, tau)) {                     // not among the vectors: ties too
                    const int at = atomicAdd(&sh.n, 1);
                    if (at < CAP) sh.list[at] = cand_key(zs, lp + (unsigned)ch.single);
                }
                for (;;) {
                    auto put = [&](int i, const u32x4 (&q)[BAT]) {
                        const int at = atomicAdd(&sh.slots, 1);
                        if (at >= SLOTS) return;
#pragma unroll
                        for (int k = 0; k < BAT; ++k) sh.batch[at][k] = q[k];
                        sh.from[at] = (unsigned)(i * BAT * NT + tid);
                        hit &= ~(1u << i);
                    };
                    if (KEEP) {
#pragma unroll
                        for (int i = 0; i < NB; ++i)
                            if (hit >> i & 1) put(i, raw[i]);
                    } else {
#pragma unroll 1
                        for (unsigned h = hit; h; h &= h - 1) {
                            const int i = __ffs(h) - 1;
                            u32x4 q[BAT];
                            load(i, q);
                            mask(i, q);
                            put(i, q);
                        }
                    }
                    __syncthreads();
                    const int slots = sh.slots;
                    for (int x = tid; x < min(slots, SLOTS) * NE; x += NT) {
                        const int at = x / NE, j = x % NE;
                        const float z = load1<BF>(sh.batch[at], j);
                        if (take(z)) {
                            const int o = atomicAdd(&sh.n, 1);
                            const unsigned e = (sh.from[at] + (unsigned)(j / V * NT)) * V + (unsigned)(j % V);
                            if (o < CAP) sh.list[o] = cand_key(z, l0 + e);
                        }
                    }
                    __syncthreads();
                    if (slots <= SLOTS || sh.n > CAP) return;       // all of them, or too many anyway
                    __syncthreads();
                    if (tid == 0) sh.slots = 0;
                    __syncthreads();
                }
            };
            gather(true);
            if (sh.n > CAP) {
                // Very many logits equal to tau: those above it, and of the
                // equal ones the first of the first K threads that have any, in
                // label order (vector by vector, thread by thread).
                __syncthreads();
                if (tid == 0) sh.n = sh.slots = 0;
                __syncthreads();
                gather(false);
                int found = 0;
                for (int i0 = 0; i0 < ch.cnt && found < a.K; i0 += NT) {
                    unsigned set = 0;
                    if (i0 + tid < ch.cnt) {
                        const u32x4 q = ch.p[i0 + tid];
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float z = elem<BF>(q, j);
                            set |= (z == tau && is_cand(z) ? 1u : 0u) << j;
                        }
                    }
                    const unsigned long long have = __ballot(set != 0);
                    if ((tid & 63) == 0) sh.u[tid >> 6] = (unsigned)__popcll(have);
                    __syncthreads();
                    int before = __popcll(have & ((1ull << (tid & 63)) - 1)), all = 0;
#pragma unroll
                    for (int i = 0; i < NT / 64; ++i) {
                        before += i < tid >> 6 ? (int)sh.u[i] : 0;
                        all += (int)sh.u[i];
                    }
                    if (set && found + before < a.K) {
                        int at = atomicAdd(&sh.n, __popc(set));
                        for (; set; set &= set - 1, ++at)
                            if (at < CAP) sh.list[at] = cand_key(tau, l0 + (unsigned)(i0 + tid) * V + (__ffs(set) - 1));
                    }
                    found += all;
                    __syncthreads();
                }
                __syncthreads();
            }
            if (sh.n <= CAP) {
                rank_keys(sh, sh.n, a.K);
            } else {
                // Very many logits above tau in a few threads: the best one
                // below the last, K times.
                key_t last = ~(key_t)0;
                for (int q = 0; q < a.K; ++q) {
                    key_t best = is_cand(zs) ? cand_key(zs, lp + (unsigned)ch.single) : 0;
                    if (best >= last) best = 0;
#pragma unroll 1
                    for (int i = tid; i < ch.cnt; i += NT) {
                        const u32x4 t = ch.p[i];
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float z = elem<BF>(t, j);
                            const key_t x = is_cand(z) ? cand_key(z, l0 + (unsigned)i * V + j) : 0;
                            if (x < last && x > best) best = x;
                        }
                    }
                    last = block_max(best, sh.key);
                    if (tid == 0) sh.top[q] = last;
                }
                __syncthreads();
            }
        }
        if (ONE) {
            finish_row<BF>(a, b, st, given, sh, w.loss);
        } else {
            if (tid == 0) w.stat[item] = st;
            if (tid < a.K) w.key[(int64_t)item * a.K + tid] = sh.top[tid];
        }
        __syncthreads();      // the next item's use of sh
    }
}

// A row's chunks joined, one workgroup a row.  Latency counts (7.3 us for 512
// rows, 5.0 for one row of 527 chunks): all that can be is loaded first, only the
// chunks' best keys are compared, and the other keys of those few chunks that can
// hold one of the row's best are read after that.
template <bool BF>
__global__ __launch_bounds__(NT) void k_lp_rows(LogprobArgs a, Cut cut) {
    __shared__ Shared sh;
    const int nc = cut.chunks();
    const Ws w = ws_map(a, cut.items);
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (threadIdx.x == 0) sh.n = 0;
        // statistics and best key of the chunks; memory first, waits after
        const key_t *key = w.key + b * nc * a.K;
        constexpr int SB = 4;             // chunks a thread at a time
        Stat s[SB];
        key_t first[SB];
        auto fetch = [&](int c0) {
#pragma unroll
            for (int q = 0; q < SB; ++q) {
                const int c = c0 + q * NT, at = min(c, nc - 1);
                s[q] = w.stat[b * nc + at];
                first[q] = a.K > 0 ? key[(int64_t)at * a.K] : 0;
                if (c >= nc) {
                    s[q] = (Stat){kNegInf, 0.f, 0.f};
                    first[q] = 0;
                }
            }
        };
        fetch(threadIdx.x);
        const Given given = read_given<BF>(a, b);
        Stat st = {kNegInf, 0.f, 0.f};
        unsigned best = 0;
        for (int c0 = threadIdx.x;;) {
            const Stat both[2] = {st, stat_join(s)};
            st = stat_join(both);
#pragma unroll
            for (int q = 0; q < SB; ++q) best = max(best, (unsigned)(first[q] >> 32));
            c0 += SB * NT;
            if (c0 >= nc) break;
            fetch(c0);
        }
        kth_put(best, sh);
        st = block_join(st, sh.st);       // its barrier publishes sh.best and sh.n too
        if (a.K > 0) {
            // a value that K keys reach (0: fewer, everything); a chunk's keys that
            // reach it, which lie in order
            const key_t t = max((key_t)kth_get(a.K, sh) << 32, (key_t)1);
            for (int c0 = threadIdx.x; c0 < nc; c0 += SB * NT) {
                if (nc > SB * NT) fetch(c0);          // else they are here already
                unsigned hit = 0;
#pragma unroll
                for (int q = 0; q < SB; ++q) hit |= (first[q] >= t ? 1u : 0u) << q;
#pragma unroll 1
                for (; hit; hit &= hit - 1) {
                    const key_t *from = key + (int64_t)(c0 + (__ffs(hit) - 1) * NT) * a.K;
                    key_t k[8];
                    int n = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) k[j] = j < a.K ? from[j] : 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) n += k[j] >= t ? 1 : 0;
                    const int at = atomicAdd(&sh.n, n);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n && at + j < CAP) sh.list[at + j] = k[j];
                }
            }
            __syncthreads();
            if (sh.n <= CAP) {
                rank_keys(sh, sh.n, a.K);
            } else {
                key_t last = ~(key_t)0;
                for (int q = 0; q < a.K; ++q) {
                    key_t next = 0;
                    for (int i = threadIdx.x; i < nc * a.K; i += NT)
                        if (key[i] < last && key[i] > next) next = key[i];
                    last = block_max(next, sh.key);
                    if (threadIdx.x == 0) sh.top[q] = last;
                }
                __syncthreads();
            }
        }
        finish_row<BF>(a, b, st, given, sh, w.loss);
        __syncthreads();
    }
}

// *loss += s * the sum of the rows' losses, in a fixed order
__global__ __launch_bounds__(NT) void k_lp_loss(LogprobArgs a, Cut cut) {
    __shared__ float sl[NT / 64];
    const Ws w = ws_map(a, cut.items);
    float t = 0.f;
    for (int b = threadIdx.x; b < a.B; b += NT) t += w.loss[b];
    t = wave_sum_dpp(t);
    if ((threadIdx.x & 63) == 0) sl[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) *a.loss += a.s * (sl[0] + sl[1] + sl[2] + sl[3]);
}

template <bool BF>
static hipError_t launch_fwd(const LogprobArgs &a, hipStream_t st) {
    const Cut cut = cut_rows(a.B, a.n[0], a.n[1], a.bf);
    const unsigned most = 1u << 22;
    const dim3 grid((unsigned)(cut.items < most ? cut.items : most)), rows((unsigned)(a.B < (1 << 22) ? a.B : 1 << 22));
    if (!cut.covered()) return hipErrorInvalidValue;      // a kernel that would leave logits out
#define GO(ONE) \
    if (cut.nb == 1) hipLaunchKernelGGL((k_lp_stats<BF, 1, ONE>), grid, dim3(NT), 0, st, a, cut); \
    else if (cut.nb == 2) hipLaunchKernelGGL((k_lp_stats<BF, 2, ONE>), grid, dim3(NT), 0, st, a, cut); \
    else if (cut.nb == 4) hipLaunchKernelGGL((k_lp_stats<BF, 4, ONE>), grid, dim3(NT), 0, st, a, cut); \
    else hipLaunchKernelGGL((k_lp_stats<BF, 8, ONE>), grid, dim3(NT), 0, st, a, cut)
    if (cut.chunks() == 1) {
        GO(true);
    } else {
        GO(false);
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
// are added by rewriting their elements after the barrier.  All of a thread's
// eight loads are under way before the row's scalars are read: 512 x 670,192
// bf16 with entropy 250 us, 5.5 TB/s, as fast as a copy (264 us at 5.2 TB/s).
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
            G = wave_sum_dpp(G);
            if ((tid & 63) == 0) sg[tid >> 6] = G;
            __syncthreads();
            G = sg[0] + sg[1] + sg[2] + sg[3];
            __syncthreads();      // the next item's use of sg
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
