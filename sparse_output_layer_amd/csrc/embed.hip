// embed.hip -- embedding bags: weighted sums of table rows, and the table's
// gradient by sorted tokens.
//
//   y[b]  = s sum_{e in row b} w_e E[t_e]
//   dE[v] = s sum_{e: t_e = v} w_e dy[row e],   dw_e = s <E[t_e], dy[row e]>
//
// Both sums are one operation: a list of entries ordered by the row they are
// added to, each a coefficient and a row to read.  Bags come in that order;
// for the gradient the entries are sorted by token (stable, so that a token's
// entries are added in the order of the list).  The list is cut into chunks of
// equal numbers of entries, whatever the rows' lengths are: frequent tokens
// and long documents do not make a thread's share longer.  A sum that lies in
// one chunk is written at once; the parts of one that goes over chunks are
// left in the workspace and added in their order by k_seg_join.  No atomics on
// floating-point values: equal inputs give equal bits.
#include "rows.h"

#include <type_traits>

namespace haste {

namespace {

constexpr int NT = 256;

// the row of a CSR list that entry e lies in (rows may be empty), or -1
__device__ __forceinline__ int row_of(const int32_t *row_ptr, int B, int e) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (row_ptr[mid] <= e) lo = mid;
        else hi = mid;
    }
    return row_ptr[lo] <= e && e < row_ptr[lo + 1] ? lo : -1;
}

// the eight values of a row's vector, added to, in fp32
template <bool BF>
__device__ __forceinline__ void put_row8(void *p, int64_t i, int c, int D, bool add, const float *a) {
    float v[8];
    if (add) {
        load8n<BF>(p, i, c, D, 0.f, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += a[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = a[j];
    }
    store8n<BF>(p, i, D - c, v);
}

}  // namespace

// ------------------------------------------------- one token a row: a copy
// TPR threads a row, a vector of eight columns each (blockIdx.y takes the
// columns past 8 TPR); a workgroup's threads load U rows before they store
// them.  Rows of a table larger than the caches come from anywhere in memory:
// what counts is the number of them under way.  65536 rows of 1024 bf16 from a table
// of 205 MB: 44 us, 5.5 TB/s (4 rows a thread instead of 8: 49).
template <bool EB, bool YB, int TPR>
__global__ __launch_bounds__(NT) void k_embed_lookup(EmbedArgs a) {
    constexpr int RW = NT / TPR, U = EB ? 8 : 4;
    const int g = threadIdx.x / TPR, c = 8 * ((int)blockIdx.y * TPR + (int)threadIdx.x % TPR);
    const bool tail = a.D & 7;
    if (c >= a.D) return;
    for (int64_t r0 = (int64_t)blockIdx.x * RW * U + g; r0 < a.B; r0 += (int64_t)gridDim.x * RW * U) {
        int tok[U];
        float w[U];
        Raw8<EB> v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t r = r0 + i * RW;
            const int t = r < a.B ? a.tok[r] : -1;
            tok[i] = t >= 0 && t < a.V ? t : -1;
            w[i] = a.scale * (a.w && r < a.B ? a.w[r] : 1.f);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = raw8n<EB>(a.E, tok[i] < 0 ? 0 : (int64_t)tok[i] * a.D + c, c, tok[i] < 0 ? 0 : a.D, tail);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t r = r0 + i * RW;
            if (r >= a.B) break;
            float x[8];
            unpack8n<EB>(v[i], c, tok[i] < 0 ? 0 : a.D, tail, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = tok[i] < 0 ? 0.f : x[j] * w[i];
            store8n<YB>(a.y, r * a.D + c, a.D - c, x);
        }
    }
}

// ------------------------------------------------------ few entries: bags
// A workgroup a row and 64 vectors, its WV waves a share of the row's entries
// each: one launch, no workspace.
template <bool EB, bool YB, int WV>
__global__ __launch_bounds__(64 * WV) void k_embed_rows(EmbedArgs a) {
    __shared__ float part[WV][64 * 9];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = 8 * (64 * (int)blockIdx.y + lane);
    const bool tail = a.D & 7;
    const int b = blockIdx.x;
    const int e0 = max(0, a.row_ptr[b]), e1 = min(a.n, a.row_ptr[b + 1]);
    float s[8] = {};
    constexpr int U = 8;
    for (int e = e0 + w; e < e1; e += WV * U) {
        Raw8<EB> r[U];
        float k[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = e + WV * i;
            int tok = at < e1 ? a.tok[at] : -1;
            if (tok >= a.V) tok = -1;
            k[i] = tok < 0 ? 0.f : a.scale * (a.w ? a.w[at] : 1.f);
            r[i] = raw8n<EB>(a.E, tok < 0 ? 0 : (int64_t)tok * a.D + c, c, tok < 0 ? 0 : a.D, tail);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float x[8];
            unpack8n<EB>(r[i], c, a.D, tail, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = __builtin_fmaf(k[i], x[j], s[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[w][9 * lane + j] = s[j];
    __syncthreads();
    // a thread's columns: the waves' parts in their order
    for (int i = threadIdx.x; i < 512 && 512 * (int)blockIdx.y + i < a.D; i += 64 * WV) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < WV; ++k) t += part[k][9 * (i >> 3) + (i & 7)];
        store1<YB>(a.y, (int64_t)b * a.D + 512 * (int)blockIdx.y + i, t);
    }
}

// --------------------------------------------- sums over an ordered list
// TPR threads a chunk of C entries, a vector of eight columns each; blockIdx.y
// takes the columns past 8 TPR.  SORTED: the list is that of the sort;
// otherwise the bags' own, and the workgroups past the chunks' write the rows
// that have no entries.  EW (0 none, 1 bf16, 2 fp32): an entry's row is also
// multiplied with the row of E that its sum belongs to, the weights' gradient:
// a token's row of E is then read once for its entries of a chunk, and rows of
// `in` not a second time.  60,007 fp32 entries of 768 with the weights' gradient 36
// to 50 us (E's rows from the caches or not), 65536 bf16 ones of 1024 26 to 34.
template <bool SB, bool DB, bool SORTED, int EW, int TPR>
__global__ __launch_bounds__(NT) void k_seg_sum(SegArgs a) {
    constexpr int RW = NT / TPR, C = kSegChunk, WAVES = TPR > 64 ? TPR / 64 : 1;
    __shared__ int dst[RW][C + 2], src[RW][C];
    __shared__ float co[RW][C];
    __shared__ int ids[EW ? RW : 1][C];
    __shared__ float dot[EW ? RW : 1][WAVES][C];
    const int g = threadIdx.x / TPR, li = threadIdx.x % TPR, c = 8 * ((int)blockIdx.y * TPR + li);
    const bool tail = a.D & 7;
    if (!SORTED && (int64_t)blockIdx.x * RW >= a.chunks) {
        const int64_t blocks = (a.chunks + RW - 1) / RW;
        const float zero[8] = {};
        for (int64_t b = ((int64_t)blockIdx.x - blocks) * RW + g; b < a.rows; b += (gridDim.x - blocks) * RW)
            if (a.row_ptr[b] >= a.row_ptr[b + 1] && c < a.D) store8n<DB>(a.out, b * a.D + c, a.D - c, zero);
        return;
    }
    const int64_t chunk = (int64_t)blockIdx.x * RW + g, e0 = chunk * C;
    const int cnt = (int)max((int64_t)0, min((int64_t)C, a.n - e0));
    // dst[i + 1] = the row entry i is added to, with the entries before and after the chunk
    for (int i = li; i < C + 2; i += TPR) {
        const int64_t e = e0 + i - 1;
        int d = -1;
        if (chunk < a.chunks && e >= 0 && e < a.n && i <= cnt + 1) {
            const bool mine = i >= 1 && i <= cnt;
            if (SORTED) {
                d = a.dst[e];
                if (mine) {
                    const int id = a.id[e];
                    const int f = d < 0 ? -1 : a.row ? a.row[id] : id;
                    src[g][i - 1] = f;
                    co[g][i - 1] = f < 0 ? 0.f : a.scale * (a.w ? a.w[id] : 1.f);
                    if (EW) ids[g][i - 1] = id;
                }
            } else {
                d = row_of(a.row_ptr, a.rows, (int)e);
                if (mine) {
                    int tok = a.tok[e];
                    if (tok >= a.V) tok = -1;
                    src[g][i - 1] = tok < 0 ? -1 : tok;
                    co[g][i - 1] = tok < 0 ? 0.f : a.scale * (a.w ? a.w[e] : 1.f);
                }
            }
        }
        dst[g][i] = d;
    }
    __syncthreads();
    const int before = dst[g][0], after = dst[g][cnt + 1], head = dst[g][1], last = dst[g][cnt];
    if (li == 0 && blockIdx.y == 0 && cnt > 0) {
        a.head[chunk] = head;
        a.last[chunk] = last;
    }
    if (!EW && (cnt == 0 || c >= a.D)) return;
    float *part = a.part + chunk * 2 * a.D;
    float s[8] = {};
    int cur = head;
    bool begun = before == head;            // the sum began in the chunk before
    // a sum's end: written, or a part of it left for k_seg_join
    auto flush = [&](bool goes_on) {
        if (cur < 0 || (EW && c >= a.D)) return;
        if (begun) store8n<false>(part, c, a.D - c, s);
        else if (goes_on) store8n<false>(part, a.D + c, a.D - c, s);
        else put_row8<DB>(a.out, (int64_t)cur * a.D + c, c, a.D, a.accumulate, s);
    };
    // more rows under way gain nothing (fp32 with the weights' gradient, 60,007
    // entries of 768: 4 at a time 50 us, 8 at a time or 4 and 4 in turn 61)
    constexpr int U = SB ? 8 : 4;
    for (int i0 = 0; i0 < cnt; i0 += U) {
        Raw8<SB> r[U];
        Raw8<EW == 1> ev[EW ? U : 1];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int f = i0 + i < cnt ? src[g][i0 + i] : -1;
            r[i] = raw8n<SB>(a.in, f < 0 ? 0 : (int64_t)f * a.D + c, c, f < 0 ? 0 : a.D, tail);
            if (EW) {
                const int t = f < 0 ? -1 : dst[g][i0 + i + 1];
                ev[EW ? i : 0] = raw8n<EW == 1>(a.E, t < 0 ? 0 : (int64_t)t * a.D + c, c, t < 0 ? 0 : a.D, tail);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i0 + i >= cnt) break;
            const int d = dst[g][i0 + i + 1], D = src[g][i0 + i] < 0 ? 0 : a.D;
            if (d != cur) {
                flush(false);
                begun = false;
                cur = d;
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = 0.f;
            }
            float x[8];
            unpack8n<SB>(r[i], c, D, tail, x);
            const float k = co[g][i0 + i];
            if (D) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = __builtin_fmaf(k, x[j], s[j]);
            }
            if (EW) {
                float y[8], p = 0.f;
                unpack8n<EW == 1>(ev[EW ? i : 0], c, D, tail, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) p = __builtin_fmaf(x[j], y[j], p);
                float none[2][NT / 64];
                int turn = 0;
                p = TPR <= 64 ? row_sum<(TPR <= 64 ? TPR : 64), NT>(p, none, turn) : wave_sum_dpp(p);
                if ((li & 63) == 0) dot[g][li / 64][i0 + i] = p;
            }
        }
    }
    flush(after == last);
    if (!EW) return;
    __syncthreads();
    for (int i = li; i < cnt; i += TPR) {
        float p = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) p += dot[g][w][i];
        a.dw[ids[g][i]] = dst[g][i + 1] < 0 || src[g][i] < 0 ? 0.f : a.scale * p;
    }
}

// A sum that began in chunk b and goes on: its part there and those of the
// chunks after it that begin with the same row, in their order.  A workgroup
// takes 16 chunks and 256 columns, a wave one chunk: most begin no such sum.  One of up to kLong
// parts is added up by its wave; longer ones by all 16 waves after that, a
// sixteenth of the parts each, joined in LDS.
constexpr int kLong = 12;
template <bool DB>
__device__ __forceinline__ void seg_out(const SegArgs &a, int row, int c, int m, const float *s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < m) {
            const int64_t o = (int64_t)row * a.D + c + j;
            store1<DB>(a.out, o, a.accumulate ? load1<DB>(a.out, o) + s[j] : s[j]);
        }
}
// four columns of the parts w, w + step, ... of a sum that begins in chunk b
__device__ __forceinline__ void seg_parts(const SegArgs &a, int64_t b, int n, int w, int step, int c, int m, float *s) {
    constexpr int U = 6;
    for (int i0 = w; i0 <= n; i0 += U * step) {
        f32x4 t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            // the first part is the chunk's second slot, the others' are first slots
            const float *p = a.part + ((b + i) * 2 + (i == 0)) * a.D + c;
            t[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if (i <= n) {
                if (m >= 4) {
                    t[u] = *(const f32x4u *)p;
                } else {
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (j < m) t[u][j] = p[j];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += t[u][j];
    }
}
template <bool DB>
__global__ __launch_bounds__(1024) void k_seg_join(SegArgs a) {
    __shared__ float part[16][64][5];
    __shared__ int count[16];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t b = (int64_t)blockIdx.x * 16 + w;
    const int c = 256 * (int)blockIdx.y + 4 * lane;
    int n = 0;                               // parts after the first
    if (b + 1 < a.chunks) {
        const int row = a.last[b];
        // it goes on, and did not begin before
        if (row >= 0 && a.head[b + 1] == row && !(a.head[b] == row && b > 0 && a.last[b - 1] == row)) {
            for (;;) {
                const int64_t at = b + 1 + n + lane;
                const uint64_t same = __ballot(at < a.chunks && a.head[at] == row);
                const int run = ~same ? __builtin_ctzll(~same) : 64;
                n += run;
                if (run < 64) break;
            }
            if (n < kLong && c < a.D) {
                float s[4] = {};
                seg_parts(a, b, n, 0, 1, c, a.D - c, s);
                seg_out<DB>(a, row, c, a.D - c, s);
            }
        }
    }
    if (lane == 0) count[w] = n;
    __syncthreads();
    for (int i = 0; i < 16; ++i) {
        const int m = count[i];
        if (m < kLong) continue;
        const int64_t f = (int64_t)blockIdx.x * 16 + i;
        float s[4] = {};
        if (c < a.D) seg_parts(a, f, m, w, 16, c, a.D - c, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) part[w][lane][j] = s[j];
        __syncthreads();
        if (w == 0 && c < a.D) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) s[j] += part[k][lane][j];
            }
            seg_out<DB>(a, a.last[f], c, a.D - c, s);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- the sort
// Least significant digit first, stable, up to 1024 digits a pass.  A
// workgroup counts a run of entries, then places them: every workgroup adds
// up the counts of all of them itself (at most kSortBlocks rows of counts), so
// that a pass is two launches (60,007 entries: 7.7 and 12 us, the gradient's zeros
// among it).  Keys are tokens; those outside the table get
// the key V, past all others.
constexpr int ST = 512, SW = ST / 64;

constexpr int SU = 4;      // loads of a thread under way together: the sort's workgroups are few and wait for memory
// the keys of entries e, e + step, ... (past the end of the list its last one's)
__device__ __forceinline__ void sort_keys(const SortArgs &a, int64_t e, int step, int *key) {
    const int *p = a.first ? a.tok : a.key_in;
#pragma unroll
    for (int i = 0; i < SU; ++i) key[i] = p[min(e + i * step, a.n - 1)];
#pragma unroll
    for (int i = 0; i < SU; ++i) key[i] = a.first && (key[i] < 0 || key[i] >= a.V) ? a.V : key[i];
}

// Beside the sort, whose few workgroups wait for memory most of the time: the
// zeros of the gradient's rows (134 MB: 19 us alone) and the entries' rows.
__device__ __forceinline__ void sort_beside(const SortArgs &a, int block, int blocks) {
    const int64_t at = (int64_t)block * ST + threadIdx.x, step = (int64_t)blocks * ST;
    if (a.row)
        for (int64_t e = at; e < a.n; e += step) a.row[e] = row_of(a.row_ptr, a.B, (int)e);
    const int64_t n = (a.z1 - a.z0) / 16;
    char *p = a.zero + a.z0;
    for (int64_t i = at; i < n; i += step) *(u32x4h *)(p + 16 * i) = (u32x4){0u, 0u, 0u, 0u};
    if (at < (a.z1 - a.z0 - 16 * n) / 2) ((unsigned short *)(p + 16 * n))[at] = 0;
}

__global__ __launch_bounds__(ST) void k_sort_count(SortArgs a) {
    if ((int)blockIdx.x >= a.blocks) {
        sort_beside(a, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    __shared__ int cnt[1024];
    const int bins = 1 << a.bits;
    for (int i = threadIdx.x; i < bins; i += ST) cnt[i] = 0;
    __syncthreads();
    const int64_t e0 = blockIdx.x * a.run, e1 = min(a.n, e0 + a.run);
    for (int64_t e = e0 + threadIdx.x; e < e1; e += SU * ST) {
        int key[SU];
        sort_keys(a, e, ST, key);
#pragma unroll
        for (int i = 0; i < SU; ++i)
            if (e + i * ST < e1) atomicAdd(&cnt[(key[i] >> a.shift) & (bins - 1)], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += ST) a.hist[(int64_t)blockIdx.x * bins + i] = cnt[i];
}

__global__ __launch_bounds__(ST) void k_sort_place(SortArgs a) {
    if ((int)blockIdx.x >= a.blocks) {
        sort_beside(a, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    __shared__ int cnt[SW][1024];
    __shared__ int wsum[SW];
    const int bins = 1 << a.bits, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < bins; i += ST)
        for (int k = 0; k < SW; ++k) cnt[k][i] = 0;
    __syncthreads();
    // the wave's own run of entries, counted
    const int64_t per = (a.run + SW - 1) / SW, b0 = blockIdx.x * a.run, b1 = min(a.n, b0 + a.run);
    const int64_t e0 = min(b1, b0 + w * per), e1 = min(b1, e0 + per);
    for (int64_t e = e0 + lane; e < e1; e += SU * 64) {
        int key[SU];
        sort_keys(a, e, 64, key);
#pragma unroll
        for (int i = 0; i < SU; ++i)
            if (e + i * 64 < e1) atomicAdd(&cnt[w][(key[i] >> a.shift) & (bins - 1)], 1);
    }
    // digits' totals, and those of the workgroups before: thread t the digits 2t, 2t + 1
    int total[2] = {0, 0}, mine[2] = {0, 0};
    if (2 * tid < bins) {
        constexpr int U = 16;
        for (int b0 = 0; b0 < a.blocks; b0 += U) {
            u32x2 v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = *(const u32x2 *)(a.hist + (int64_t)min(b0 + i, a.blocks - 1) * bins + 2 * tid);
            __builtin_amdgcn_sched_barrier(0);      // all of them before the first is waited for
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    total[k] += b0 + i < a.blocks ? (int)v[i][k] : 0;
                    mine[k] += b0 + i < (int)blockIdx.x ? (int)v[i][k] : 0;
                }
        }
    }
    // exclusive scan over the digits
    const int both = total[0] + total[1];
    int scan = both;
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(scan, o, 64);
        if (lane >= o) scan += t;
    }
    if (lane == 63) wsum[w] = scan;
    __syncthreads();
    int base = scan - both;
    for (int i = 0; i < w; ++i) base += wsum[i];
    // the waves' first places
    for (int k = 0; k < 2; ++k) {
        const int d = 2 * tid + k;
        if (d < bins) {
            int at = base + mine[k] + (k ? total[0] : 0);
            for (int i = 0; i < SW; ++i) {
                const int v = cnt[i][d];
                cnt[i][d] = at;
                at += v;
            }
        }
    }
    __syncthreads();
    volatile int *place = cnt[w];
    for (int64_t r = e0 + lane; r - lane < e1; r += SU * 64) {
        int keys[SU], id[SU];
        sort_keys(a, r, 64, keys);
#pragma unroll
        for (int i = 0; i < SU; ++i) id[i] = a.first ? (int)(r + i * 64) : a.id_in[min(r + i * 64, a.n - 1)];
#pragma unroll
        for (int u = 0; u < SU; ++u) {
            const bool live = r + u * 64 < e1;
            const int key = keys[u], d = (key >> a.shift) & (bins - 1);
            uint64_t same = __ballot(live);
            for (int i = 0; i < a.bits; ++i) {
                const uint64_t one = __ballot(d >> i & 1);
                same &= (d >> i & 1) ? one : ~one;
            }
            const int below = __popcll(same & ((1ull << lane) - 1));
            int at = 0;
            if (live) at = place[d] + below;
            __builtin_amdgcn_wave_barrier();
            if (live && (same >> lane) == 1) place[d] = at + 1;       // the last of its digit
            __builtin_amdgcn_wave_barrier();
            if (live) {
                a.key_out[at] = a.last && key >= a.V ? -1 : key;
                a.id_out[at] = id[u];
            }
        }
    }
}

// ------------------------------------------------- the weights' gradient
// <E[t], dy[row]> of eight consecutive entries a wave, their table rows on
// their way together; a bag's entries share its row of dy.
template <bool EB, bool YB>
__global__ __launch_bounds__(NT) void k_embed_dw(EmbedArgs a) {
    constexpr int U = 8;
    const int lane = threadIdx.x & 63;
    const bool tail = a.D & 7;
    for (int64_t e0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * U; e0 < a.n; e0 += (int64_t)gridDim.x * 4 * U) {
        // lane i < 8 finds entry i's token and row
        int tok = -1, row = -1;
        if (lane < U && e0 + lane < a.n) {
            tok = a.tok[e0 + lane];
            row = a.row_ptr ? row_of(a.row_ptr, a.B, (int)(e0 + lane)) : (int)(e0 + lane);
            if (tok < 0 || tok >= a.V || row < 0) tok = row = -1;
        }
        int t[U], r[U];
        bool one = true;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            t[i] = __builtin_amdgcn_readlane(tok, i);
            r[i] = __builtin_amdgcn_readlane(row, i);
            one = one && r[i] == r[0];
        }
        float s[U] = {};
        for (int c0 = 0; c0 < a.D; c0 += 512) {      // 512 columns' sums one after another, as k_seg_sum forms them
            const int c = c0 + 8 * lane;
            Raw8<EB> x[U];
#pragma unroll
            for (int i = 0; i < U; ++i) x[i] = raw8n<EB>(a.E, t[i] < 0 ? 0 : (int64_t)t[i] * a.D + c, c, t[i] < 0 ? 0 : a.D, tail);
            float g[8];
            auto load = [&](int i) {
                unpack8n<YB>(raw8n<YB>(a.dy, r[i] < 0 ? 0 : (int64_t)r[i] * a.D + c, c, r[i] < 0 ? 0 : a.D, tail), c, r[i] < 0 ? 0 : a.D, tail, g);
            };
            load(0);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (!one && i) load(i);
                float v[8], p = 0.f;
                unpack8n<EB>(x[i], c, t[i] < 0 ? 0 : a.D, tail, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) p = __builtin_fmaf(g[j], v[j], p);
                s[i] += wave_sum_dpp(p);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (lane == i && e0 + i < a.n) a.dw[e0 + i] = t[i] < 0 ? 0.f : a.scale * s[i];
    }
}

// zeros in 16-byte pieces, and the elements past the last
__global__ __launch_bounds__(NT) void k_embed_zero(void *p, int64_t bytes) {
    const int64_t n = bytes / 16, stride = (int64_t)gridDim.x * NT;
    int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i < (bytes & 15) / 2) ((unsigned short *)p)[n * 8 + i] = 0;
    for (; i < n; i += stride) *(u32x4h *)((char *)p + 16 * i) = (u32x4){0u, 0u, 0u, 0u};
}

namespace {

int64_t seg_chunks(int64_t n) { return (n + kSegChunk - 1) / kSegChunk; }
inline size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// of n entries and sums of D columns: parts, the chunks' first and last rows
size_t seg_bytes(int64_t n, int D) {
    const size_t c = (size_t)seg_chunks(n);
    return up(c * 2 * (size_t)D * 4) + 2 * up(c * 4);
}
void seg_place(SegArgs &s, char *ws) {
    const size_t c = (size_t)s.chunks;
    s.part = (float *)ws;
    s.head = (int *)(ws + up(c * 2 * (size_t)s.D * 4));
    s.last = (int *)((char *)s.head + up(c * 4));
}

template <bool SB, bool DB, bool SORTED, int EW>
hipError_t seg_sum(const SegArgs &a, hipStream_t st) {
    // the rows without entries: as many workgroups as write them in few turns
    auto go = [&](int tpr) {
        const int rw = NT / tpr;
        int64_t x = (a.chunks + rw - 1) / rw;
        if (!SORTED) {
            const int64_t z = ((int64_t)a.rows + rw - 1) / rw;
            x += z < 1024 ? z : 1024;
        }
        return dim3((unsigned)x, (unsigned)((a.D + 8 * tpr - 1) / (8 * tpr)));
    };
#define GO(T) hipLaunchKernelGGL((k_seg_sum<SB, DB, SORTED, EW, T>), go(T), dim3(NT), 0, st, a)
    if (a.D <= 128) GO(16);
    else if (a.D <= 256) GO(32);
    else if (a.D <= 512) GO(64);
    else if (a.D <= 1024) GO(128);
    else GO(256);
#undef GO
    if (a.chunks)
        hipLaunchKernelGGL((k_seg_join<DB>), dim3((unsigned)((a.chunks + 15) / 16), (unsigned)((a.D + 255) / 256)), dim3(1024), 0, st, a);
    return hipGetLastError();
}
template <bool SORTED, int EW>
hipError_t seg_sum_any(const SegArgs &a, bool sb, bool db, hipStream_t st) {
    if (sb && db) return seg_sum<true, true, SORTED, EW>(a, st);
    if (sb) return seg_sum<true, false, SORTED, EW>(a, st);
    if (db) return seg_sum<false, true, SORTED, EW>(a, st);
    return seg_sum<false, false, SORTED, EW>(a, st);
}
// columns of a workgroup of k_seg_sum at most
constexpr int kSegWidth = 2048;

// Bags by one launch, a workgroup each, or as a list cut into chunks.  A long bag
// keeps its workgroup alone: one bag of 512 entries (768 bf16 columns) takes 13 us
// against 18, of 1024 24 against 19; 16 bags of 512 in all 8 against 18.  Of up to
// kWideBags bags each has 16 waves (the bag of 512 with four: 39 us; 64 short bags
// 8.1 against 7.7, 512 of them 10 against 7.5).
constexpr int kFewEntries = 768, kWideBags = 256;
constexpr int kFewBags = 1 << 20;     // a workgroup each, and a launch has fewer than 2^32 threads
bool few(int B, int n) { return n <= kFewEntries && B <= kFewBags; }
constexpr int kSortBlocks = 128;

struct SortPlan {
    int passes, bits, blocks;
    int64_t run;
};
SortPlan sort_plan(int64_t n, int V) {
    SortPlan p;
    int bits = 1;
    while (bits < 31 && (V >> bits) != 0) ++bits;        // keys 0 .. V
    p.passes = (bits + 9) / 10;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.run = (n + kSortBlocks - 1) / kSortBlocks;
    if (p.run < 2048) p.run = 2048;
    p.blocks = (int)((n + p.run - 1) / p.run);
    return p;
}

}  // namespace

size_t embed_fwd_ws_bytes(bool bags, int B, int n, int D) {
    return bags && !few(B, n) ? seg_bytes(n, D) : 0;
}

hipError_t launch_embed_fwd(const EmbedArgs &a, hipStream_t st) {
    if (!a.row_ptr) {
        auto go = [&](auto eb, auto yb) {
            auto launch = [&](auto tpr) {
                constexpr int T = decltype(tpr)::value, per = NT / T * (decltype(eb)::value ? 8 : 4);
                const int64_t x = ((int64_t)a.B + per - 1) / per;
                hipLaunchKernelGGL((k_embed_lookup<decltype(eb)::value, decltype(yb)::value, T>),
                                   dim3((unsigned)(x < 65536 ? x : 65536), (unsigned)((a.D + 8 * T - 1) / (8 * T))), dim3(NT), 0, st, a);
            };
            if (a.D <= 128) launch(std::integral_constant<int, 16>{});
            else if (a.D <= 512) launch(std::integral_constant<int, 64>{});
            else launch(std::integral_constant<int, 128>{});
        };
        const std::true_type bf;
        const std::false_type f32;
        if (a.ebf && a.ybf) go(bf, bf);
        else if (a.ebf) go(bf, f32);
        else if (a.ybf) go(f32, bf);
        else go(f32, f32);
        return hipGetLastError();
    }
    if (few(a.B, a.n)) {
        const dim3 grid(a.B, (unsigned)(((int64_t)a.D + 511) / 512));
        auto go = [&](auto eb, auto yb) {
            constexpr bool E = decltype(eb)::value, Y = decltype(yb)::value;
            if (a.B <= kWideBags) hipLaunchKernelGGL((k_embed_rows<E, Y, 16>), grid, dim3(1024), 0, st, a);
            else hipLaunchKernelGGL((k_embed_rows<E, Y, 4>), grid, dim3(NT), 0, st, a);
        };
        const std::true_type bf;
        const std::false_type f32;
        if (a.ebf && a.ybf) go(bf, bf);
        else if (a.ebf) go(bf, f32);
        else if (a.ybf) go(f32, bf);
        else go(f32, f32);
        return hipGetLastError();
    }
    SegArgs s{};
    s.in = a.E;
    s.out = a.y;
    s.row_ptr = a.row_ptr;
    s.tok = a.tok;
    s.w = a.w;
    s.n = a.n;
    s.chunks = seg_chunks(a.n);
    s.rows = a.B;
    s.D = a.D;
    s.V = a.V;
    s.scale = a.scale;
    seg_place(s, (char *)a.ws);
    return seg_sum_any<false, 0>(s, a.ebf, a.ybf, st);
}

size_t embed_bwd_ws_bytes(int n, int V, int D) {
    if (n == 0) return 0;
    const SortPlan p = sort_plan(n, V);
    return seg_bytes(n, D) + 5 * up((size_t)n * 4) + up((size_t)p.blocks * 1024 * 4);
}

hipError_t launch_embed_bwd(const EmbedArgs &a, hipStream_t st) {
    const int64_t bytes = a.dE && !a.accumulate ? (int64_t)a.V * a.D * (a.gbf ? 2 : 4) : 0;
    if (bytes && a.n == 0) {
        const int64_t want = (bytes / 16 + NT) / NT;
        hipLaunchKernelGGL(k_embed_zero, dim3((unsigned)(want < 16384 ? want : 16384)), dim3(NT), 0, st, a.dE, bytes);
    }
    if (a.n == 0) return hipGetLastError();
    const bool with = a.dE && a.dw && a.D <= kSegWidth;      // the weights' gradient in the sums' pass
    if (a.dw && !with) {
        const int64_t want = ((int64_t)a.n + 31) / 32;
        const dim3 grid((unsigned)(want < 65536 ? want : 65536));
#define GO(E, Y) hipLaunchKernelGGL((k_embed_dw<E, Y>), grid, dim3(NT), 0, st, a)
        if (a.ebf && a.ybf) GO(true, true);
        else if (a.ebf) GO(true, false);
        else if (a.ybf) GO(false, true);
        else GO(false, false);
#undef GO
    }
    if (!a.dE) return hipGetLastError();
    const SortPlan p = sort_plan(a.n, a.V);
    char *ws = (char *)a.ws + seg_bytes(a.n, a.D);
    const size_t nb = up((size_t)a.n * 4);
    int *key[2] = {(int *)ws, (int *)(ws + nb)}, *id[2] = {(int *)(ws + 2 * nb), (int *)(ws + 3 * nb)};
    SortArgs t{};
    t.tok = a.tok;
    t.row_ptr = a.row_ptr;
    t.hist = (int *)(ws + 5 * nb);
    t.n = a.n;
    t.B = a.B;
    t.V = a.V;
    t.bits = p.bits;
    t.run = p.run;
    t.blocks = p.blocks;
    t.zero = (char *)a.dE;
    int *row = a.row_ptr ? (int *)(ws + 4 * nb) : nullptr;
    const int launches = 2 * p.passes;
    const int64_t share = (bytes / launches + 255) / 256 * 256;
    for (int i = 0; i < launches; ++i) {
        t.first = i < 2;
        t.last = i >= launches - 2;
        t.shift = i / 2 * p.bits;
        t.key_in = key[(i / 2 + 1) & 1];
        t.id_in = id[(i / 2 + 1) & 1];
        t.key_out = key[i / 2 & 1];
        t.id_out = id[i / 2 & 1];
        t.row = i == 0 ? row : nullptr;
        t.z0 = i * share < bytes ? i * share : bytes;
        t.z1 = i + 1 == launches || (i + 1) * share > bytes ? bytes : (i + 1) * share;
        // workgroups beside the sort: for 64 KB of zeros each, or for the rows, at most two a CU
        int64_t beside = (t.z1 - t.z0 + 65535) / 65536;
        if (t.row && beside < (a.n + ST - 1) / ST) beside = (a.n + ST - 1) / ST;
        const dim3 grid((unsigned)(p.blocks + (beside < 512 ? beside : 512)));
        if (i % 2 == 0) hipLaunchKernelGGL(k_sort_count, grid, dim3(ST), 0, st, t);
        else hipLaunchKernelGGL(k_sort_place, grid, dim3(ST), 0, st, t);
    }
    SegArgs s{};
    s.in = a.dy;
    s.out = a.dE;
    s.dst = t.key_out;
    s.id = t.id_out;
    s.row = row;
    s.w = a.w;
    s.scale = a.scale;
    s.n = a.n;
    s.chunks = seg_chunks(a.n);
    s.rows = a.V;
    s.D = a.D;
    s.accumulate = a.accumulate;
    seg_place(s, (char *)a.ws);
    if (!with) return seg_sum_any<true, 0>(s, a.ybf, a.gbf, st);
    s.E = a.E;
    s.dw = a.dw;
    return a.ebf ? seg_sum_any<true, 1>(s, a.ybf, a.gbf, st) : seg_sum_any<true, 2>(s, a.ybf, a.gbf, st);
}

}  // namespace haste
