// Group norm with an activation over the rows of each graph of a batch,
// channels last.  Graph i owns rows seg[i] .. seg[i + 1] - 1; a group is D
// adjacent columns; the statistics run over all rows of the graph and all
// columns of the group:
//   xhat = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  Out = act(xhat w + v)
// and with a = act'(xhat w + v) G, h = a w, n values in the group:
//   dw = sum a xhat, dv = sum a (over all rows of all graphs);
//   dX = rstd (h - sum(h) / n - xhat sum(h xhat) / n).
//
// Bound: HBM.  The rows are cut into chunks of equal length, one workgroup
// each, whatever the graphs' lengths.  A graph short enough for the registers
// of a workgroup (8 rows a thread: 64 rows of 256 bf16 columns) is done whole
// by the chunk it starts in, in one read and one write.  A longer one is met
// in pieces: chunk c and graph g meet in at most one piece, and the pieces in
// row order are a staircase, so piece (c, g) is number c + g: every piece has
// a place of its own without a plan, and a graph's pieces are neighbours.  A
// second kernel joins a graph's pieces in piece order (in 64 bits) and a third
// pass over the long graphs applies them.
// The statistics do not lose the variance to a large mean: a thread sums its
// rows' differences from its first row and their squares, and the group's
// squares are then taken about the group's mean (Chan, Golub and LeVeque's
// pairwise formula).  Where the first row is itself an outlier at distance D,
// a thread of n rows loses n D^2 2^-24 of squares that hold D^2.
#include <type_traits>

#include "drop.h"
#include "ops.h"
#include "trace.h"

namespace sag {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kHold = 4;              // rows a thread holds at once
constexpr int64_t kMaxChunks = 2048, kMaxGraphBlocks = 2048;   // eight workgroups a CU each
constexpr int kShort = 32;            // a graph of so many rows a thread is one workgroup's

struct NormArgs {
    const void* x;
    int64_t ldx, n_rows, d;
    int groups, gd;               // columns per group
    const int64_t* seg;           // null: one graph of all rows
    int64_t n_seg;
    const float* w;               // null: 1
    const float* v;               // null: 0
    float eps, slope;
    float* mean;
    float* rstd;
    void* out;                    // forward: Out; backward: dX
    int64_t ldo;
    const void* g;                // backward
    int64_t ldg;
    float2* piece;                // [n_chunks + n_seg][groups]
    float2* stat;                 // backward: [n_seg][groups] means of h and h xhat
    float* col;                   // backward: [graph_blocks + chunk_blocks][2][d] column sums
    int64_t rows_per_chunk, n_chunks;
    int64_t short_rows;           // graphs of up to so many rows are done whole
    int64_t graph_blocks;         // the first pass's workgroups for short graphs, before the chunks'
    int64_t seg_per_block;        // graphs and groups per block of the joining kernel
    int grp_per_block;
    int tx, ty;                   // threads across the columns' vectors and down the rows
};

__device__ __forceinline__ int64_t seg_at(const NormArgs& a, int64_t i) {
    if (!a.seg) return i == 0 ? 0 : a.n_rows;
    const int64_t s = a.seg[i];
    return s < 0 ? 0 : (s > a.n_rows ? a.n_rows : s);
}

// Last graph that starts at or before row r, by 64 probes a step (all lanes
// of every wavefront return the same value); -1: r lies before the first.
__device__ __forceinline__ int64_t seg_of(const NormArgs& a, int64_t r) {
    if (!a.seg) return 0;
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, n = a.n_seg + 1;          // the answer + 1 lies in [lo, lo + n]
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t i = lo + (lane + 1) * step - 1;
        const bool le = i < lo + n && seg_at(a, i) <= r;
        const int cnt = __popcll(__ballot(le));
        const int64_t nlo = lo + cnt * step;
        const int64_t left = lo + n - nlo;
        lo = nlo;
        n = left < step - 1 ? left : step - 1;
        if (n < 0) n = 0;
    }
    return lo - 1;
}

// Calls f(graph, first row, end row, piece) for each piece of a long graph
// (over short_rows rows) in this chunk, the same for every thread of the
// workgroup (all of them have to take part).  The lanes look at 64 graphs at
// a time, so a chunk of short ones costs three loads in a row.
template <class F>
__device__ __forceinline__ void for_pieces(const NormArgs& a, int64_t chunk, F&& f) {
    const int64_t r0 = chunk * a.rows_per_chunk;
    const int64_t end = r0 + a.rows_per_chunk < a.n_rows ? r0 + a.rows_per_chunk : a.n_rows;
    const int lane = threadIdx.x & 63;
    int64_t g0 = seg_of(a, r0);
    if (g0 < 0) g0 = 0;
    while (g0 < a.n_seg) {
        const int64_t g = g0 + lane;
        const bool in = g < a.n_seg;
        const int64_t gs = in ? seg_at(a, g) : a.n_rows, ge = in ? seg_at(a, g + 1) : a.n_rows;
        uint64_t todo = __ballot(ge - gs > a.short_rows && gs < end && ge > r0);
        while (todo) {
            const int i = __ffsll(static_cast<unsigned long long>(todo)) - 1;
            todo &= todo - 1;
            const int64_t is = __shfl(gs, i, 64), ie = __shfl(ge, i, 64);
            const int64_t lo = is > r0 ? is : r0, hi = ie < end ? ie : end;
            f(g0 + i, lo, hi, chunk + g0 + i);
        }
        if (__ballot(gs >= end)) break;
        g0 += 64;
    }
}

__device__ __forceinline__ uint4 as_uint4(u32x4_t v) { return make_uint4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ u32x4_t load16(const void* p) { return *reinterpret_cast<const u32x4_t*>(p); }
template <class T>
__device__ __forceinline__ void unpack_vec(u32x4_t v, float (&f)[Vec<T>::N]) { unpack<T>(as_uint4(v), f); }

// Rows r, r + ty, ... below hi (a piece has fewer than 2^31).
__device__ __forceinline__ uint32_t rows_of(const NormArgs& a, int64_t r, int64_t hi) {
    return r < hi ? static_cast<uint32_t>(hi - r - 1) / static_cast<uint32_t>(a.ty) + 1u : 0u;
}

// f(vectors of x and, with TWO, of y) for the `cnt` rows of a thread, `sx`
// (`sy`) bytes apart, four rows' loads at a time.  Pointers only ever move by
// the step, and rows past the last cost no arithmetic: a graph of 25 rows is
// short enough for address products and selects to take longer than its data.
template <bool TWO, class F>
__device__ __forceinline__ void each_row(const void* x, int64_t sx, const void* y, int64_t sy, int64_t cnt, F&& f) {
    const char* px = static_cast<const char*>(x);
    const char* py = static_cast<const char*>(y);
    for (; cnt >= kHold; cnt -= kHold) {
        u32x4_t q[kHold], g[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            q[i] = load16(px);
            px += sx;
            if constexpr (TWO) {
                g[i] = load16(py);
                py += sy;
            }
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) f(q[i], g[i]);
    }
    if (cnt > 0) {
        u32x4_t q[kHold - 1], g[kHold - 1];
#pragma unroll
        for (int i = 0; i < kHold - 1; ++i) {
            q[i] = load16(px);
            if constexpr (TWO) g[i] = load16(py);
            if (i + 1 < cnt) {
                px += sx;
                py += sy;
            }
        }
#pragma unroll
        for (int i = 0; i < kHold - 1; ++i)
            if (i < cnt) f(q[i], g[i]);
    }
}

// ---- sums over the rows and columns of a group, by the whole workgroup -----------------
// A thread owns one 16-byte vector of columns.  Where whole vectors lie in
// one group (gd a multiple of V) it brings one value a sum, else one a
// column; `n` of these slots make a row of threads.
struct Slots {
    int n, per_group;
};

template <bool COL>
__host__ __device__ inline Slots slots_of(int64_t d, int gd, int tx, int V) {
    return COL ? Slots{static_cast<int>(d), gd} : Slots{tx, gd / V};
}

// out[k][group] (LDS) = sum over the group of v[k][column] of every thread
// that is `on`.  sh: [N][ty][slots].  Every thread of the workgroup takes
// part; `out` is visible to all after the call, and sh may be written again.
template <int N, int V, bool COL>
__device__ __forceinline__ void group_sums(const NormArgs& a, const Slots& sl, bool on, int tx, int ty, int nc,
                                           const float (&v)[N][V], float* sh, float* out) {
    const int plane = a.ty * sl.n;
    if (on) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (COL) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < nc) sh[k * plane + ty * sl.n + tx * V + e] = v[k][e];
            } else {
                float s = v[k][0];
#pragma unroll
                for (int e = 1; e < V; ++e) s += v[k][e];
                sh[k * plane + ty * sl.n + tx] = s;
            }
        }
    }
    __syncthreads();
    // a power of two of lanes to a group, each taking every lpg-th value
    int lpg = 1;
    while (lpg < 64 && 2 * lpg * a.groups <= kThreads) lpg *= 2;
    const int gl = threadIdx.x & (lpg - 1), gpp = kThreads / lpg, vals = a.ty * sl.per_group;
    const float inv = 1.f / static_cast<float>(sl.per_group);
    for (int gb = 0; gb < a.groups; gb += gpp) {
        const int gi = gb + static_cast<int>(threadIdx.x) / lpg;
        const bool ok = gi < a.groups;
        float s[N];
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = 0.f;
        if (ok) {
            for (int i = gl; i < vals; i += lpg) {
                // i = r * per_group + c (below 2^12: the quotient is exact after one step)
                int r = static_cast<int>(static_cast<float>(i) * inv);
                int c = i - r * sl.per_group;
                if (c < 0) { --r; c += sl.per_group; }
                if (c >= sl.per_group) { ++r; c -= sl.per_group; }
#pragma unroll
                for (int k = 0; k < N; ++k) s[k] += sh[k * plane + r * sl.n + gi * sl.per_group + c];
            }
        }
        for (int o = 1; o < lpg; o *= 2)
#pragma unroll
            for (int k = 0; k < N; ++k) s[k] += __shfl_xor(s[k], o, 64);
        if (ok && gl == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) out[k * a.groups + gi] = s[k];
    }
    __syncthreads();
}

// This thread's columns: the affine and, per graph, the statistics (one of
// each where the vector lies in one group, else one a column).
template <int V, bool COL>
struct Cols {
    static constexpr int G = COL ? V : 1;
    float w[V], v[V], mean[G], rstd[G];
    int grp[G];
    static __device__ __forceinline__ constexpr int of(int e) { return COL ? e : 0; }
    __device__ __forceinline__ void init(const NormArgs& a, int c0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = c0 + e < a.d ? c0 + e : static_cast<int>(a.d) - 1;
            w[e] = a.w ? a.w[c] : 1.f;
            v[e] = a.v ? a.v[c] : 0.f;
            if (e < G) grp[e] = c / a.gd;
        }
    }
    __device__ __forceinline__ void graph(const NormArgs& a, int64_t g) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            mean[i] = a.mean[g * a.groups + grp[i]];
            rstd[i] = a.rstd[g * a.groups + grp[i]];
        }
    }
};

template <class T, int ACT, bool COL>
__device__ __forceinline__ void norm_store(T* p, u32x4_t q, const Cols<Vec<T>::N, COL>& k,
                                           const float (&rw)[Vec<T>::N], float slope, int nc) {
    constexpr int V = Vec<T>::N;
    float f[V];
    unpack_vec<T>(q, f);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = act_value<ACT, T>(fmaf(f[e] - k.mean[k.of(e)], rw[e], k.v[e]), slope);
    store_first<T>(p, f, nc);
}

// The first `cnt` of the thread's rows from x on: Out from X.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void apply_rows(const T* x, int64_t sx, T* out, int64_t so, int64_t cnt,
                                           const Cols<Vec<T>::N, COL>& k, const float (&rw)[Vec<T>::N], float slope,
                                           int nc) {
    char* po = reinterpret_cast<char*>(out);
    each_row<false>(x, sx, nullptr, 0, cnt, [&](u32x4_t q, u32x4_t) {
        norm_store<T, ACT, COL>(reinterpret_cast<T*>(po), q, k, rw, slope, nc);
        po += so;
    });
}

// ---- forward ----------------------------------------------------------------------------
// First pass: workgroups below graph_blocks do short graphs whole (and give
// graphs without rows their statistics), the others take the chunks' pieces
// of long graphs: mean and squares about it.
template <class T, int ACT, bool COL>
__global__ __launch_bounds__(kThreads, 4) void norm_first(NormArgs a) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __attribute__((aligned(16))) float sh[];
    const Slots sl = slots_of<COL>(a.d, a.gd, a.tx, V);
    float* gsum = sh + a.ty * sl.n;       // [groups]
    float* gsq = gsum + a.groups;         // [groups]
    const int tx = threadIdx.x % a.tx, ty = threadIdx.x / a.tx;
    const bool on = ty < a.ty;
    const int c0 = tx * V;
    const int nc = a.d - c0 < V ? static_cast<int>(a.d) - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    T* out = static_cast<T*>(a.out) + c0;
    Cols<V, COL> k;
    k.init(a, c0);
    const int64_t sx = a.ty * a.ldx * static_cast<int64_t>(sizeof(T)), so = a.ty * a.ldo * static_cast<int64_t>(sizeof(T));
    // the group means (k.mean, and gsum / total) and squares about them (gsq) of rows lo .. hi - 1
    auto stats = [&](int64_t lo, int64_t hi) {
        const uint32_t cnt = on ? rows_of(a, lo + ty, hi) : 0u;
        const float n = static_cast<float>(cnt);
        float m[V], s[V], c[V];
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] = s[e] = c[e] = 0.f;
        if (cnt) {
            const T* xr = x + (lo + ty) * a.ldx;
            unpack_vec<T>(load16(xr), c);
            each_row<false>(xr, sx, nullptr, 0, cnt, [&](u32x4_t q, u32x4_t) {
                float f[V];
                unpack_vec<T>(q, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float t = f[e] - c[e];
                    m[e] += t;
                    s[e] = fmaf(t, t, s[e]);
                }
            });
            const float inv = 1.f / n;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float t = m[e] * inv;
                s[e] = fmaxf(fmaf(-t, m[e], s[e]), 0.f);
                m[e] = c[e] + t;
            }
        }
        const float itot = 1.f / (static_cast<float>(hi - lo) * static_cast<float>(a.gd));
        float v[1][V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[0][e] = e < nc ? m[e] * n : 0.f;
        group_sums<1, V, COL>(a, sl, on, tx, ty, nc, v, sh, gsum);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (e < k.G) k.mean[e] = gsum[k.grp[e]] * itot;
            const float dm = m[e] - k.mean[k.of(e)];
            v[0][e] = e < nc ? s[e] + dm * dm * n : 0.f;
        }
        group_sums<1, V, COL>(a, sl, on, tx, ty, nc, v, sh, gsq);
        // (gsum and gsq stay until the next call's first barrier)
        return itot;
    };
    if (blockIdx.x < a.graph_blocks) {
        for (int64_t g = blockIdx.x; g < a.n_seg; g += a.graph_blocks) {
            const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
            if (hi - lo > a.short_rows) continue;
            if (hi <= lo) {
                for (int i = threadIdx.x; i < a.groups; i += kThreads) {
                    a.mean[g * a.groups + i] = 0.f;
                    a.rstd[g * a.groups + i] = 1.f / sqrtf(a.eps);
                }
                continue;
            }
            const float itot = stats(lo, hi);
            for (int i = threadIdx.x; i < a.groups; i += kThreads) {
                a.mean[g * a.groups + i] = gsum[i] * itot;
                a.rstd[g * a.groups + i] = __builtin_amdgcn_rsqf(gsq[i] * itot + a.eps);
            }
            float rw[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (e < k.G) k.rstd[e] = __builtin_amdgcn_rsqf(gsq[k.grp[e]] * itot + a.eps);
                rw[e] = k.rstd[k.of(e)] * k.w[e];
            }
            // (every row is read before it is written, by the same thread)
            apply_rows<T, ACT, COL>(x + (lo + ty) * a.ldx, sx, out + (lo + ty) * a.ldo, so,
                                    on ? rows_of(a, lo + ty, hi) : 0u, k, rw, a.slope, nc);
        }
    } else {
        for_pieces(a, static_cast<int64_t>(blockIdx.x) - a.graph_blocks, [&](int64_t, int64_t lo, int64_t hi, int64_t piece) {
            const float itot = stats(lo, hi);
            for (int i = threadIdx.x; i < a.groups; i += kThreads)
                a.piece[piece * a.groups + i] = make_float2(gsum[i] * itot, gsq[i]);
        });
    }
}

// Joins the pieces of long graphs per group.  A block has seg_per_block graphs and grp_per_block
// groups; threads are groups (a power of two) by parts, each part taking every
// parts-th piece, and the parts are added in a fixed tree.  BWD: the pieces
// hold sums of h and h xhat.
template <bool BWD>
__global__ __launch_bounds__(kThreads) void norm_join(NormArgs a) {
    __shared__ double p0[kThreads], p1[kThreads];
    const int64_t s_lo = static_cast<int64_t>(blockIdx.x) * a.seg_per_block;
    const int64_t s_hi = s_lo + a.seg_per_block < a.n_seg ? s_lo + a.seg_per_block : a.n_seg;
    const int g_lo = static_cast<int>(blockIdx.y) * a.grp_per_block;
    const int g_hi = g_lo + a.grp_per_block < a.groups ? g_lo + a.grp_per_block : a.groups;
    int gw = 1;
    while (gw < kThreads && gw < g_hi - g_lo) gw *= 2;
    const int parts = kThreads / gw, part = threadIdx.x / gw, gl = threadIdx.x % gw;
    for (int64_t g = s_lo; g < s_hi; ++g) {
        const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
        if (hi - lo <= a.short_rows) continue;
        const int64_t first = lo / a.rows_per_chunk, last = (hi - 1) / a.rows_per_chunk;
        const double n = static_cast<double>(hi - lo) * a.gd;
        for (int gb = g_lo; gb < g_hi; gb += gw) {
            const int gi = gb + gl;
            double s0 = 0.0, s1 = 0.0, c = 0.0;
            if (gi < g_hi) {
                const float2* q = a.piece + g * a.groups + gi;
                if constexpr (!BWD) c = q[first * a.groups].x;
#pragma unroll 4
                for (int64_t k = first + part; k <= last; k += parts) {
                    const float2 v = q[k * a.groups];
                    if constexpr (BWD) {
                        s0 += v.x;
                        s1 += v.y;
                    } else {
                        const int64_t b = k * a.rows_per_chunk, e = b + a.rows_per_chunk;
                        const double nk = static_cast<double>((e < hi ? e : hi) - (b > lo ? b : lo)) * a.gd;
                        const double dm = v.x - c;
                        s0 += nk * dm;
                        s1 += v.y + nk * dm * dm;
                    }
                }
            }
            p0[threadIdx.x] = s0;
            p1[threadIdx.x] = s1;
            __syncthreads();
            for (int o = parts / 2; o > 0; o /= 2) {
                if (part < o) {
                    p0[threadIdx.x] += p0[threadIdx.x + o * gw];
                    p1[threadIdx.x] += p1[threadIdx.x + o * gw];
                }
                __syncthreads();
            }
            if (part == 0 && gi < g_hi) {
                s0 = p0[threadIdx.x];
                s1 = p1[threadIdx.x];
                if constexpr (BWD) {
                    a.stat[g * a.groups + gi] = make_float2(static_cast<float>(s0 / n), static_cast<float>(s1 / n));
                } else {
                    const double dm = s0 / n;
                    double var = s1 / n - dm * dm;
                    if (var < 0.0) var = 0.0;
                    a.mean[g * a.groups + gi] = static_cast<float>(c + dm);
                    a.rstd[g * a.groups + gi] = static_cast<float>(1.0 / sqrt(var + static_cast<double>(a.eps)));
                }
            }
            __syncthreads();
        }
    }
}

template <class T, int ACT, bool COL>
__global__ __launch_bounds__(kThreads, 4) void norm_apply(NormArgs a) {
    constexpr int V = Vec<T>::N;
    const int tx = threadIdx.x % a.tx;
    // (a thread past the last row of threads walks along with no rows: the
    // search for a row's graph takes whole wavefronts)
    const int ty = threadIdx.x / a.tx;
    const bool on = ty < a.ty;
    const int c0 = tx * V;
    const int nc = a.d - c0 < V ? static_cast<int>(a.d) - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    T* out = static_cast<T*>(a.out) + c0;
    Cols<V, COL> k;
    k.init(a, c0);
    // the last chunks first: they are what the first pass left in the caches
    for_pieces(a, a.n_chunks - 1 - static_cast<int64_t>(blockIdx.x), [&](int64_t g, int64_t lo, int64_t hi, int64_t) {
        k.graph(a, g);
        float rw[V];
#pragma unroll
        for (int e = 0; e < V; ++e) rw[e] = k.rstd[k.of(e)] * k.w[e];
        if (!on || lo + ty >= hi) return;
        apply_rows<T, ACT, COL>(x + (lo + ty) * a.ldx, a.ty * a.ldx * static_cast<int64_t>(sizeof(T)), out + (lo + ty) * a.ldo,
                                a.ty * a.ldo * static_cast<int64_t>(sizeof(T)), rows_of(a, lo + ty, hi), k, rw, a.slope, nc);
    });
}

// ---- backward ---------------------------------------------------------------------------
// a = act'(z) g of one element, and xhat.  ReLU's and leaky ReLU's step at
// z = 0 is taken where the formula's z changes sign, not where one rounding
// of it does: with d = x - mean = dh + dl and rstd w = rh + rl (each the
// rounded value and what the rounding left), z = fma(dh, rh, v) + (dh rl + dl
// rh) is right to about 2^-46 of its terms, for seven operations more.
template <int ACT>
struct Affine {           // rstd w of a column
    float rh, rl;
    __device__ __forceinline__ Affine(float rstd, float w) : rh(rstd * w), rl(0.f) {
        if constexpr (ACT == SAG_ACT_RELU || ACT == SAG_ACT_LEAKY_RELU) rl = fmaf(rstd, w, -rh);
    }
};

template <int ACT>
__device__ __forceinline__ float grad_a(float x, float g, float mean, float rstd, const Affine<ACT>& k, float v,
                                        float slope, float& xhat) {
    const float dh = x - mean;
    xhat = dh * rstd;
    float z = fmaf(dh, k.rh, v);
    if constexpr (ACT == SAG_ACT_RELU || ACT == SAG_ACT_LEAKY_RELU) {
        const float b = dh - x;                                  // Knuth's two-sum
        const float dl = (x - (dh - b)) - (mean + b);
        z += fmaf(dh, k.rl, dl * k.rh);
    }
    return times_act_grad<ACT>(g, z, slope);
}

// dX of one vector from the means m0 of h and m1 of h xhat.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void norm_dx_store(T* p, u32x4_t qx, u32x4_t qg, const Cols<Vec<T>::N, COL>& k,
                                              const float (&m0)[Cols<Vec<T>::N, COL>::G],
                                              const float (&m1)[Cols<Vec<T>::N, COL>::G], float slope, int nc) {
    constexpr int V = Vec<T>::N;
    float f[V], q[V];
    unpack_vec<T>(qx, f);
    unpack_vec<T>(qg, q);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float xh;
        const int i = k.of(e);
        const float t = grad_a<ACT>(f[e], q[e], k.mean[i], k.rstd[i], Affine<ACT>(k.rstd[i], k.w[e]), k.v[e], slope, xh);
        f[e] = k.rstd[i] * (t * k.w[e] - m0[i] - xh * m1[i]);
    }
    store_first<T>(p, f, nc);
}

// The thread's rows lo + ty, lo + 2 ty, ... below hi: dX.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void dx_rows(const NormArgs& a, int c0, int64_t r, int64_t hi,
                                        const Cols<Vec<T>::N, COL>& k, const float (&m0)[Cols<Vec<T>::N, COL>::G],
                                        const float (&m1)[Cols<Vec<T>::N, COL>::G], int nc) {
    constexpr int64_t ES = sizeof(T);
    char* po = reinterpret_cast<char*>(static_cast<T*>(a.out) + r * a.ldo + c0);
    each_row<true>(static_cast<const T*>(a.x) + r * a.ldx + c0, a.ty * a.ldx * ES,
                   static_cast<const T*>(a.g) + r * a.ldg + c0, a.ty * a.ldg * ES, rows_of(a, r, hi),
                   [&](u32x4_t qx, u32x4_t qg) {
                       norm_dx_store<T, ACT, COL>(reinterpret_cast<T*>(po), qx, qg, k, m0, m1, a.slope, nc);
                       po += a.ty * a.ldo * ES;
                   });
}

// First pass: dX of short graphs whole (when wanted), the pieces' sums of h
// and h xhat of long ones, and each workgroup's column sums of a and a xhat.
template <class T, int ACT, bool COL>
__global__ __launch_bounds__(kThreads, COL ? 2 : 3) void norm_bwd_first(NormArgs a) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __attribute__((aligned(16))) float sh[];
    const Slots sl = slots_of<COL>(a.d, a.gd, a.tx, V);
    const int d = static_cast<int>(a.d);
    float* acc = sh + 2 * a.ty * sl.n;    // [2][ty][d]: the sums of a and a xhat, each thread its own
    float* gsum = acc + 2 * a.ty * d;     // [2][groups]
    const int tx = threadIdx.x % a.tx, ty = threadIdx.x / a.tx;
    const bool on = ty < a.ty;
    const int c0 = tx * V;
    const int nc = d - c0 < V ? d - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    const T* gr = static_cast<const T*>(a.g) + c0;
    T* out = static_cast<T*>(a.out) + c0;
    Cols<V, COL> k;
    k.init(a, c0);
    float* acc0 = acc + ty * d + c0;
    float* acc1 = acc0 + a.ty * d;
    if (on)
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nc) acc0[e] = acc1[e] = 0.f;
    // (piece -1: the whole of a short graph)
    auto part = [&](int64_t g, int64_t lo, int64_t hi, int64_t piece) {
        k.graph(a, g);
        float t0[V], t1[V];
#pragma unroll
        for (int e = 0; e < V; ++e) t0[e] = t1[e] = 0.f;
        if (on && lo + ty < hi)
            each_row<true>(x + (lo + ty) * a.ldx, a.ty * a.ldx * static_cast<int64_t>(sizeof(T)), gr + (lo + ty) * a.ldg,
                           a.ty * a.ldg * static_cast<int64_t>(sizeof(T)), rows_of(a, lo + ty, hi), [&](u32x4_t qx, u32x4_t qg) {
                float f[V], q[V];
                unpack_vec<T>(qx, f);
                unpack_vec<T>(qg, q);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float xh;
                    const int j = k.of(e);
                    const float t = grad_a<ACT>(f[e], q[e], k.mean[j], k.rstd[j], Affine<ACT>(k.rstd[j], k.w[e]), k.v[e],
                                                a.slope, xh);
                    t0[e] += t;
                    t1[e] = fmaf(t, xh, t1[e]);
                }
            });
        if (on)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < nc) {
                    acc0[e] += t0[e];
                    acc1[e] += t1[e];
                }
        if (!a.out) return;
        float v[2][V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[0][e] = e < nc ? t0[e] * k.w[e] : 0.f;
            v[1][e] = e < nc ? t1[e] * k.w[e] : 0.f;
        }
        group_sums<2, V, COL>(a, sl, on, tx, ty, nc, v, sh, gsum);
        if (piece >= 0) {
            for (int i = threadIdx.x; i < a.groups; i += kThreads)
                a.piece[piece * a.groups + i] = make_float2(gsum[i], gsum[a.groups + i]);
        } else {
            const float inv = 1.f / (static_cast<float>(hi - lo) * static_cast<float>(a.gd));
            float m0[k.G], m1[k.G];
#pragma unroll
            for (int e = 0; e < k.G; ++e) {
                m0[e] = gsum[k.grp[e]] * inv;
                m1[e] = gsum[a.groups + k.grp[e]] * inv;
            }
            if (on && lo + ty < hi) dx_rows<T, ACT, COL>(a, c0, lo + ty, hi, k, m0, m1, nc);
        }
    };
    if (blockIdx.x < a.graph_blocks) {
        for (int64_t g = blockIdx.x; g < a.n_seg; g += a.graph_blocks) {
            const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
            if (lo < hi && hi - lo <= a.short_rows) part(g, lo, hi, -1);
        }
    } else {
        for_pieces(a, static_cast<int64_t>(blockIdx.x) - a.graph_blocks, part);
    }
    if (a.col) {
        // the thread rows of each column, in order
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * d; c += kThreads) {
            const float* col = acc + (c < d ? c : a.ty * d + c - d);
            float s = 0.f;
            for (int r = 0; r < a.ty; ++r) s += col[r * d];
            a.col[static_cast<int64_t>(blockIdx.x) * 2 * d + c] = s;
        }
    }
}

// dv and dw: the workgroups' column sums, 8 columns by 128 parts a block, each
// part every 128th, the parts added in a fixed tree.
constexpr int kColW = 8, kColThreads = 1024;

__global__ __launch_bounds__(kColThreads) void norm_cols(const float* __restrict__ col, int64_t n_chunks, int64_t d,
                                                         float* __restrict__ dw, float* __restrict__ dv) {
    __shared__ double p[kColThreads];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kColW + threadIdx.x % kColW;   // sums of a, then of a xhat
    const int part = threadIdx.x / kColW;
    double s = 0.0;
    if (c < 2 * d) {
#pragma unroll 4
        for (int64_t k = part; k < n_chunks; k += kColThreads / kColW) s += col[k * 2 * d + c];
    }
    p[threadIdx.x] = s;
    __syncthreads();
    for (int o = kColThreads / kColW / 2; o > 0; o /= 2) {
        if (part < o) p[threadIdx.x] += p[threadIdx.x + o * kColW];
        __syncthreads();
    }
    if (part == 0 && c < 2 * d) {
        if (c < d) { if (dv) dv[c] = static_cast<float>(p[threadIdx.x]); }
        else if (dw) dw[c - d] = static_cast<float>(p[threadIdx.x]);
    }
}

template <class T, int ACT, bool COL>
__global__ __launch_bounds__(kThreads, COL ? 2 : 3) void norm_bwd_apply(NormArgs a) {
    constexpr int V = Vec<T>::N;
    const int tx = threadIdx.x % a.tx;
    const int ty = threadIdx.x / a.tx;
    const bool on = ty < a.ty;
    const int c0 = tx * V;
    const int nc = a.d - c0 < V ? static_cast<int>(a.d) - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    const T* gr = static_cast<const T*>(a.g) + c0;
    T* out = static_cast<T*>(a.out) + c0;
    Cols<V, COL> k;
    k.init(a, c0);
    for_pieces(a, a.n_chunks - 1 - static_cast<int64_t>(blockIdx.x), [&](int64_t g, int64_t lo, int64_t hi, int64_t) {
        k.graph(a, g);
        float m0[k.G], m1[k.G];
#pragma unroll
        for (int e = 0; e < k.G; ++e) {
            const float2 q = a.stat[g * a.groups + k.grp[e]];
            m0[e] = q.x;
            m1[e] = q.y;
        }
        if (on && lo + ty < hi) dx_rows<T, ACT, COL>(a, c0, lo + ty, hi, k, m0, m1, nc);
    });
}

struct Plan {
    int tx, ty;
    int64_t rows_per_chunk, n_chunks, short_rows;
    int64_t graph_blocks, chunk_blocks;   // of the first pass
};

// At most kMaxChunks chunks, of at least half a short graph.
Plan norm_plan(int64_t n_rows, int64_t d, int64_t n_seg, bool one, sag_dtype dt) {
    Plan p;
    p.tx = static_cast<int>(cdiv(d, vec_elems(dt)));
    p.ty = kThreads / p.tx;
    p.short_rows = kShort * static_cast<int64_t>(p.ty);
    p.rows_per_chunk = cdiv(n_rows, kMaxChunks);
    if (p.rows_per_chunk < p.short_rows / 2) p.rows_per_chunk = p.short_rows / 2;
    p.n_chunks = cdiv(n_rows, p.rows_per_chunk);
    // graphs are met from their lengths on the device; the host knows that no
    // graph is long when all rows make a short one, and the length of the one
    // graph of all rows
    const bool all_short = n_rows <= p.short_rows;
    p.chunk_blocks = all_short || n_seg == 0 ? 0 : p.n_chunks;
    p.graph_blocks = one && !all_short ? 0 : (n_seg < kMaxGraphBlocks ? n_seg : kMaxGraphBlocks);
    return p;
}

// The joining kernel's blocks: at most 2048 over the graphs, and with fewer
// graphs than 256 two groups each (128 parts a group).
dim3 join_grid(NormArgs& a) {
    a.seg_per_block = cdiv(a.n_seg, 2048);
    a.grp_per_block = a.n_seg < 256 && a.groups > 2 ? 2 : a.groups;
    return dim3(static_cast<unsigned>(cdiv(a.n_seg, a.seg_per_block)), static_cast<unsigned>(cdiv(a.groups, a.grp_per_block)));
}

template <class F>
void by_column(bool col, F&& f) {
    if (col) f(std::true_type{});
    else f(std::false_type{});
}

struct Ws {
    float2 *piece, *stat;
    float* col;
    size_t used;
    bool fits;
};

Ws norm_ws(const Plan& p, int64_t d, int64_t n_seg, int64_t groups, bool bwd, void* ws, size_t bytes) {
    Carver c(ws, bytes);
    Ws w{};
    w.piece = c.take<float2>((p.n_chunks + n_seg) * groups);
    if (bwd) {
        w.stat = c.take<float2>(n_seg * groups);
        w.col = c.take<float>((p.graph_blocks + p.chunk_blocks) * 2 * d);
    }
    w.used = c.used();
    w.fits = c.fits();
    return w;
}

sag_status check_norm(const std::string& who, int64_t n_rows, int64_t d, int64_t groups, const int64_t* seg, int64_t n_seg,
                      sag_act act, float slope, sag_dtype dt) {
    if (dt != SAG_F32 && dt != SAG_BF16) return fail(SAG_E_INVALID, who + ": bad dtype");
    if (n_rows < 0 || n_seg < 0 || d < 1) return fail(SAG_E_INVALID, who + ": bad size");
    if (groups < 1 || d % groups) return fail(SAG_E_INVALID, who + ": groups must divide the width");
    if (!seg && n_seg != 1) return fail(SAG_E_INVALID, who + ": null seg with other than one graph");
    if (!act_ok(act)) return fail(SAG_E_INVALID, who + ": unknown activation");
    if (!std::isfinite(slope)) return fail(SAG_E_INVALID, who + ": slope not finite");
    if (d > 256 * vec_elems(dt)) return fail(SAG_E_UNSUPPORTED, who + ": width above 1024 (fp32) or 2048 (bf16)");
    if (n_seg >= (1 << 24)) return fail(SAG_E_UNSUPPORTED, who + ": 2^24 graphs or more");
    return SAG_OK;
}

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" size_t sag_group_norm_forward_workspace_bytes(int64_t n_rows, int64_t d, int64_t groups, int64_t n_seg,
                                                         sag_dtype dt) {
    if (n_rows < 0 || d < 1 || groups < 1 || n_seg < 0 || (dt != SAG_F32 && dt != SAG_BF16) || d > 256 * vec_elems(dt)) return 0;
    return norm_ws(norm_plan(n_rows, d, n_seg, false, dt), d, n_seg, groups, false, nullptr, 0).used;
}

extern "C" sag_status sag_group_norm_forward(const void* X, int64_t ldx, int64_t n_rows, int64_t d, int64_t groups,
                                             const int64_t* seg, int64_t n_seg, const float* w, const float* b,
                                             float eps, sag_act act, float slope, sag_dtype dt, void* Out, int64_t ldo,
                                             float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
    const std::string who = "group_norm forward";
    SAG_TRY(check_norm(who, n_rows, d, groups, seg, n_seg, act, slope, dt));
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(SAG_E_INVALID, who + ": eps negative or not finite");
    SAG_TRY(check_dense("group_norm X", X, n_rows, d, ldx, dt));
    SAG_TRY(check_dense("group_norm Out", Out, n_rows, d, ldo, dt));
    if (n_seg == 0) return SAG_OK;
    if (!mean || !rstd) return fail(SAG_E_INVALID, who + ": null mean or rstd");
    const Plan p = norm_plan(n_rows, d, n_seg, !seg, dt);
    const Ws q = norm_ws(p, d, n_seg, groups, false, ws, ws_bytes);
    if (!ws || !aligned16(ws) || !q.fits) return fail(SAG_E_WORKSPACE, who + ": workspace too small");
    hipStream_t s = static_cast<hipStream_t>(stream);
    TraceScope trace(trace_enabled() ? shape_name("group_norm", dt == SAG_BF16 ? "bf16" : "f32", n_rows, d, groups) : std::string(),
                     s, 2 * elt_size(dt) * n_rows * d, 0);
    NormArgs a{};
    a.x = X; a.ldx = ldx; a.n_rows = n_rows; a.d = d;
    a.groups = static_cast<int>(groups); a.gd = static_cast<int>(d / groups);
    a.seg = seg; a.n_seg = n_seg; a.w = w; a.v = b; a.eps = eps; a.slope = slope;
    a.mean = mean; a.rstd = rstd; a.out = Out; a.ldo = ldo;
    a.piece = q.piece; a.rows_per_chunk = p.rows_per_chunk; a.n_chunks = p.n_chunks; a.short_rows = p.short_rows; a.graph_blocks = p.graph_blocks; a.tx = p.tx; a.ty = p.ty;
    const unsigned first = static_cast<unsigned>(p.graph_blocks + p.chunk_blocks);
    const unsigned nc = static_cast<unsigned>(p.chunk_blocks);
    const dim3 jgrid = join_grid(a);
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto tag) {
            using T = decltype(tag);
            by_column(a.gd % Vec<T>::N != 0, [&](auto cc) {
                constexpr bool COL = decltype(cc)::value;
                const size_t lds = (static_cast<size_t>(p.ty) * slots_of<COL>(d, a.gd, p.tx, Vec<T>::N).n + 2 * groups) * 4;
                norm_first<T, ACT, COL><<<first, kThreads, lds, s>>>(a);
            });
            if (!nc) return;
            norm_join<false><<<jgrid, kThreads, 0, s>>>(a);
            by_column(a.gd % Vec<T>::N != 0,
                          [&](auto cc) { norm_apply<T, ACT, decltype(cc)::value><<<nc, kThreads, 0, s>>>(a); });
        };
        if (dt == SAG_BF16) go(uint16_t{});
        else go(float{});
    });
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

extern "C" size_t sag_group_norm_backward_workspace_bytes(int64_t n_rows, int64_t d, int64_t groups, int64_t n_seg,
                                                          sag_dtype dt) {
    if (n_rows < 0 || d < 1 || groups < 1 || n_seg < 0 || (dt != SAG_F32 && dt != SAG_BF16) || d > 256 * vec_elems(dt)) return 0;
    return norm_ws(norm_plan(n_rows, d, n_seg, false, dt), d, n_seg, groups, true, nullptr, 0).used;
}

extern "C" sag_status sag_group_norm_backward(const void* X, int64_t ldx, int64_t n_rows, int64_t d, int64_t groups,
                                              const int64_t* seg, int64_t n_seg, const float* w, const float* b,
                                              sag_act act, float slope, const float* mean, const float* rstd,
                                              const void* G, int64_t ldg, float* dw, float* db, void* dX, int64_t ldd,
                                              sag_dtype dt, void* ws, size_t ws_bytes, void* stream) {
    const std::string who = "group_norm backward";
    SAG_TRY(check_norm(who, n_rows, d, groups, seg, n_seg, act, slope, dt));
    SAG_TRY(check_dense("group_norm X", X, n_rows, d, ldx, dt));
    SAG_TRY(check_dense("group_norm G", G, n_rows, d, ldg, dt));
    if (dX) SAG_TRY(check_dense("group_norm dX", dX, n_rows, d, ldd, dt));
    if (n_seg > 0 && (!mean || !rstd)) return fail(SAG_E_INVALID, who + ": null mean or rstd");
    const Plan p = norm_plan(n_rows, d, n_seg, !seg, dt);
    const Ws q = norm_ws(p, d, n_seg, groups, true, ws, ws_bytes);
    if (!ws || !aligned16(ws) || !q.fits) return fail(SAG_E_WORKSPACE, who + ": workspace too small");
    hipStream_t s = static_cast<hipStream_t>(stream);
    TraceScope trace(trace_enabled() ? shape_name("group_norm_bwd", dt == SAG_BF16 ? "bf16" : "f32", n_rows, d, groups) : std::string(),
                     s, (dX ? 3 : 2) * elt_size(dt) * n_rows * d, 0);
    NormArgs a{};
    a.x = X; a.ldx = ldx; a.n_rows = n_rows; a.d = d;
    a.groups = static_cast<int>(groups); a.gd = static_cast<int>(d / groups);
    a.seg = seg; a.n_seg = n_seg; a.w = w; a.v = b; a.slope = slope;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.out = dX; a.ldo = ldd; a.g = G; a.ldg = ldg;
    a.piece = q.piece; a.stat = q.stat; a.col = dw || db ? q.col : nullptr;
    a.rows_per_chunk = p.rows_per_chunk; a.n_chunks = p.n_chunks; a.short_rows = p.short_rows; a.graph_blocks = p.graph_blocks; a.tx = p.tx; a.ty = p.ty;
    const unsigned first = static_cast<unsigned>(p.graph_blocks + p.chunk_blocks);
    const unsigned nc = static_cast<unsigned>(p.chunk_blocks);
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto tag) {
            using T = decltype(tag);
            if (first)
                by_column(a.gd % Vec<T>::N != 0, [&](auto cc) {
                    constexpr bool COL = decltype(cc)::value;
                    const size_t lds = (static_cast<size_t>(2 * p.ty) * (d + slots_of<COL>(d, a.gd, p.tx, Vec<T>::N).n) + 2 * groups) * 4;
                    norm_bwd_first<T, ACT, COL><<<first, kThreads, lds, s>>>(a);
                });
            if (dw || db)
                norm_cols<<<static_cast<unsigned>(cdiv(2 * d, kColW)), kColThreads, 0, s>>>(q.col, first, d, dw, db);
            if (dX && nc) {
                const dim3 jgrid = join_grid(a);
                norm_join<true><<<jgrid, kThreads, 0, s>>>(a);
                by_column(a.gd % Vec<T>::N != 0,
                          [&](auto cc) { norm_bwd_apply<T, ACT, decltype(cc)::value><<<nc, kThreads, 0, s>>>(a); });
            }
        };
        if (dt == SAG_BF16) go(uint16_t{});
        else go(float{});
    });
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}
