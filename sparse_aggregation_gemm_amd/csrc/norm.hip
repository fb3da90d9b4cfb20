// Group norm with an activation over the rows of each graph of a batch,
// channels last.  Graph i owns rows seg[i] .. seg[i + 1] - 1; a group is D
// adjacent columns; the statistics run over all rows of the graph and all
// columns of the group:
//   xhat = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  Out = act(xhat w + v)
// and with a = act'(xhat w + v) G, h = a w, n values in the group:
//   dw = sum a xhat, dv = sum a (over all rows of all graphs);
//   dX = rstd (h - sum(h) / n - xhat sum(h xhat) / n).
//
// Bound: HBM (2.45M x 256 bf16 in one graph: 0.77 ms forward, 1.21 backward,
// 4.9 and 5.2 TB/s over two readings) or, for graphs of a few rows, latency.
// A short graph (kShort rows a thread) is done whole by one workgroup, or one
// wavefront, and read from HBM once.  The rows are also cut into chunks of
// equal length, a workgroup each, for the longer graphs, which are met in
// pieces: chunk c and graph g meet in at most one piece, and the pieces in row
// order are a staircase, so piece (c, g) is number c + g: every piece has a
// place of its own without a plan, and a graph's pieces are neighbours.  A
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
constexpr int kWaveHold = 16;         // rows a thread of a wavefront's graph
constexpr int64_t kManyGraphs = 512;  // from here on the shortest graphs are wavefronts'
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
    float* col;                   // backward: [the first pass's workgroups][2][d] column sums
    int64_t rows_per_chunk, n_chunks;
    int64_t short_rows;           // graphs of up to so many rows are done whole
    int64_t wave_rows;            // of these, up to so many by a wavefront
    int64_t graph_blocks, wave_blocks;   // the first pass's workgroups for short graphs; the chunks' follow
    int lanes_per_group, lanes_per_slots;   // in the sums over a group: powers of two
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

// f(vectors of x and, with TWO, of y) for the `cnt` rows of a thread, `sx`
// (`sy`) bytes apart, H rows' loads at a time.  Pointers only ever move by
// the step, and rows past the last cost no arithmetic: a graph of 25 rows is
// short enough for address products and selects to take longer than its data.
template <bool TWO, int H = kHold, class F>
__device__ __forceinline__ void each_row(const void* x, int64_t sx, const void* y, int64_t sy, int64_t cnt, F&& f) {
    const char* px = static_cast<const char*>(x);
    const char* py = static_cast<const char*>(y);
    for (; cnt >= H; cnt -= H) {
        u32x4_t q[H], g[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            q[i] = load16(px);
            px += sx;
            if constexpr (TWO) {
                g[i] = load16(py);
                py += sy;
            }
        }
#pragma unroll
        for (int i = 0; i < H; ++i) f(q[i], g[i]);
    }
    if (cnt > 0) {
        u32x4_t q[H - 1], g[H - 1];
#pragma unroll
        for (int i = 0; i < H - 1; ++i) {
            q[i] = load16(px);
            if constexpr (TWO) g[i] = load16(py);
            if (i + 1 < cnt) {
                px += sx;
                py += sy;
            }
        }
#pragma unroll
        for (int i = 0; i < H - 1; ++i)
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

// LDS for the sums per group: two planes to a team.
__host__ __device__ inline int stat_floats(const NormArgs& a) { return (a.wave_blocks ? 8 : 2) * a.groups; }

// The threads that do a graph or a piece together: a workgroup, or a
// wavefront for the shortest graphs.
template <int SZ>
struct Team {
    int tid, tx, ty, rows;      // the thread's column vector and row, and the team's rows of threads
    bool on;                    // false: past the last row of threads
    float *sums, *gs;           // LDS: [N][rows][slots], [2][groups]
    // sh: N * a.ty * slots floats for the sums, then stat_floats(a)
    __device__ __forceinline__ Team(const NormArgs& a, const Slots& sl, int n_sums, float* sh) {
        const int wave = SZ == 64 ? static_cast<int>(threadIdx.x) >> 6 : 0;
        tid = SZ == 64 ? static_cast<int>(threadIdx.x) & 63 : static_cast<int>(threadIdx.x);
        rows = SZ == 64 ? 64 / a.tx : a.ty;
        ty = static_cast<int>(static_cast<uint32_t>(tid) / static_cast<uint32_t>(a.tx));
        tx = tid - ty * a.tx;
        on = ty < rows;
        sums = sh + n_sums * wave * rows * sl.n;
        gs = sh + n_sums * a.ty * sl.n + 2 * wave * a.groups;
    }
    // Orders the team's LDS accesses before and after.
    static __device__ __forceinline__ void sync() {
        if constexpr (SZ == 64) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        } else {
            __syncthreads();
        }
    }
    // Rows lo + ty, lo + ty + rows, ... below hi (a piece has fewer than 2^31).
    __device__ __forceinline__ uint32_t count(int64_t lo, int64_t hi) const {
        return on && lo + ty < hi ? static_cast<uint32_t>(hi - lo - ty - 1) / static_cast<uint32_t>(rows) + 1u : 0u;
    }
};

// out[k][group] (LDS) = sum over the group of v[k][column] of every thread
// that is `on`.  Every thread of the team takes part; `out` is visible to all
// after the call, and t.sums may be written again.
template <int N, int V, bool COL, int SZ>
__device__ __forceinline__ void group_sums(const NormArgs& a, const Slots& sl, const Team<SZ>& t, int nc,
                                           const float (&v)[N][V], float* out) {
    const int plane = t.rows * sl.n;
    if (t.on) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (COL) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < nc) t.sums[k * plane + t.ty * sl.n + t.tx * V + e] = v[k][e];
            } else {
                float s = v[k][0];
#pragma unroll
                for (int e = 1; e < V; ++e) s += v[k][e];
                t.sums[k * plane + t.ty * sl.n + t.tx] = s;
            }
        }
    }
    t.sync();
    // a power of two of lanes to a group: across its slots, and what is left
    // of them down the rows of threads
    const int lpg = SZ == 64 ? (a.lanes_per_group > 4 ? a.lanes_per_group / 4 : 1) : a.lanes_per_group;
    const int lc = a.lanes_per_slots < lpg ? a.lanes_per_slots : lpg;
    const int shift = __builtin_ctz(lpg), cshift = __builtin_ctz(lc);
    const int gl = t.tid & (lpg - 1), g0 = t.tid >> shift, c0 = gl & (lc - 1), r0 = gl >> cshift, rs = lpg >> cshift;
    for (int gb = 0; gb < a.groups; gb += SZ >> shift) {
        const int gi = gb + g0;
        const bool ok = gi < a.groups;
        float s[N];
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = 0.f;
        if (ok) {
            const float* p = t.sums + r0 * sl.n + gi * sl.per_group;
            for (int r = r0; r < t.rows; r += rs, p += rs * sl.n)
                for (int c = c0; c < sl.per_group; c += lc)
#pragma unroll
                    for (int k = 0; k < N; ++k) s[k] += p[k * plane + c];
        }
        for (int o = 1; o < lpg; o *= 2)
#pragma unroll
            for (int k = 0; k < N; ++k) s[k] += __shfl_xor(s[k], o, 64);
        if (ok && gl == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) out[k * a.groups + gi] = s[k];
    }
    t.sync();
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
            if (e < G) grp[e] = static_cast<int>(static_cast<uint32_t>(c) / static_cast<uint32_t>(a.gd));
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

// The thread's rows of lo .. hi - 1: Out from X.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void apply_rows(const NormArgs& a, const Team<kThreads>& t, int64_t lo, int64_t hi,
                                           const Cols<Vec<T>::N, COL>& k, const float (&rw)[Vec<T>::N], int nc) {
    constexpr int64_t ES = sizeof(T);
    const uint32_t cnt = t.count(lo, hi);
    if (!cnt) return;
    const int64_t r = lo + t.ty, c0 = t.tx * Vec<T>::N;
    char* po = reinterpret_cast<char*>(static_cast<T*>(a.out) + r * a.ldo + c0);
    each_row<false>(static_cast<const T*>(a.x) + r * a.ldx + c0, t.rows * a.ldx * ES, nullptr, 0, cnt, [&](u32x4_t q, u32x4_t) {
        norm_store<T, ACT, COL>(reinterpret_cast<T*>(po), q, k, rw, a.slope, nc);
        po += t.rows * a.ldo * ES;
    });
}

// ---- forward ----------------------------------------------------------------------------
// mean and rstd of graph g out of the groups' sums and squares in t.gs, and
// the thread's rstd w.
template <int V, bool COL, int SZ>
__device__ __forceinline__ void put_stats(const NormArgs& a, const Team<SZ>& t, Cols<V, COL>& k, int64_t g, float itot,
                                          float (&rw)[V]) {
    const float* gsq = t.gs + a.groups;
    for (int i = t.tid; i < a.groups; i += SZ) {
        a.mean[g * a.groups + i] = t.gs[i] * itot;
        a.rstd[g * a.groups + i] = __builtin_amdgcn_rsqf(gsq[i] * itot + a.eps);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (e < k.G) k.rstd[e] = __builtin_amdgcn_rsqf(gsq[k.grp[e]] * itot + a.eps);
        rw[e] = k.rstd[k.of(e)] * k.w[e];
    }
}

// The group means of rows lo .. hi - 1 (k.mean; times the count in t.gs) and
// squares about them (t.gs + groups); returns 1 / the count.
template <class T, bool COL>
__device__ __forceinline__ float norm_stats(const NormArgs& a, const Slots& sl, const Team<kThreads>& t,
                                            Cols<Vec<T>::N, COL>& k, int nc, int64_t lo, int64_t hi) {
    constexpr int V = Vec<T>::N;
    const uint32_t cnt = t.count(lo, hi);
    const float n = static_cast<float>(cnt);
    float m[V], s[V], c[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = s[e] = c[e] = 0.f;
    if (cnt) {
        const T* x = static_cast<const T*>(a.x) + (lo + t.ty) * a.ldx + t.tx * V;
        unpack_vec<T>(load16(x), c);
        each_row<false>(x, t.rows * a.ldx * static_cast<int64_t>(sizeof(T)), nullptr, 0, cnt, [&](u32x4_t q, u32x4_t) {
            float f[V];
            unpack_vec<T>(q, f);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = f[e] - c[e];
                m[e] += u;
                s[e] = fmaf(u, u, s[e]);
            }
        });
        const float inv = 1.f / n;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float u = m[e] * inv;
            s[e] = fmaxf(fmaf(-u, m[e], s[e]), 0.f);
            m[e] = c[e] + u;
        }
    }
    const float itot = 1.f / (static_cast<float>(hi - lo) * static_cast<float>(a.gd));
    float v[1][V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[0][e] = e < nc ? m[e] * n : 0.f;
    group_sums<1, V, COL>(a, sl, t, nc, v, t.gs);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (e < k.G) k.mean[e] = t.gs[k.grp[e]] * itot;
        const float dm = m[e] - k.mean[k.of(e)];
        v[0][e] = e < nc ? fmaf(dm * dm, n, s[e]) : 0.f;
    }
    group_sums<1, V, COL>(a, sl, t, nc, v, t.gs + a.groups);
    // (t.gs stays until the next call's first barrier)
    return itot;
}

// Graph g of at most kWaveHold rows a thread, whole, by one wavefront that
// keeps the rows in registers: read once, summed, summed about the mean,
// written.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void norm_held(const NormArgs& a, const Slots& sl, const Team<64>& t, Cols<Vec<T>::N, COL>& k,
                                          int nc, int64_t g, int64_t lo, int64_t hi) {
    constexpr int V = Vec<T>::N, B = 4;
    const int cnt = static_cast<int>(t.count(lo, hi));
    const int steps = static_cast<int>((static_cast<uint32_t>(hi - lo) + t.rows - 1) / static_cast<uint32_t>(t.rows));   // of all lanes
    const int64_t sx = t.rows * a.ldx * static_cast<int64_t>(sizeof(T)), so = t.rows * a.ldo * static_cast<int64_t>(sizeof(T));
    const char* px = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + (cnt ? lo + t.ty : lo) * a.ldx + t.tx * V);
    u32x4_t q[kWaveHold];
#pragma unroll
    for (int b = 0; b < kWaveHold; b += B)
        if (b < steps) {
#pragma unroll
            for (int i = b; i < b + B; ++i) {
                q[i] = load16(px);
                if (i + 1 < cnt) px += sx;
            }
        }
    float v[1][V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[0][e] = 0.f;
    // (a row past the thread's last is its last again, with weight 0)
#pragma unroll
    for (int b = 0; b < kWaveHold; b += B)
        if (b < steps) {
#pragma unroll
            for (int i = b; i < b + B; ++i) {
                const float mk = i < cnt ? 1.f : 0.f;
                float f[V];
                unpack_vec<T>(q[i], f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[0][e] = fmaf(f[e], mk, v[0][e]);
            }
        }
    const float itot = 1.f / (static_cast<float>(hi - lo) * static_cast<float>(a.gd));
#pragma unroll
    for (int e = 0; e < V; ++e) v[0][e] = e < nc ? v[0][e] : 0.f;
    group_sums<1, V, COL>(a, sl, t, nc, v, t.gs);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (e < k.G) k.mean[e] = t.gs[k.grp[e]] * itot;
        v[0][e] = 0.f;
    }
    // (unpacked again: in fp32 the rows would take twice their registers)
#pragma unroll
    for (int i = 0; i < kWaveHold; ++i) asm volatile("" : "+v"(q[i]));
#pragma unroll
    for (int b = 0; b < kWaveHold; b += B)
        if (b < steps) {
#pragma unroll
            for (int i = b; i < b + B; ++i) {
                const float mk = i < cnt ? 1.f : 0.f;
                float f[V];
                unpack_vec<T>(q[i], f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float u = f[e] - k.mean[k.of(e)];
                    v[0][e] = fmaf(u * mk, u, v[0][e]);
                }
            }
        }
#pragma unroll
    for (int e = 0; e < V; ++e) v[0][e] = e < nc ? v[0][e] : 0.f;
    group_sums<1, V, COL>(a, sl, t, nc, v, t.gs + a.groups);
    float rw[V];
    put_stats(a, t, k, g, itot, rw);
#pragma unroll
    for (int i = 0; i < kWaveHold; ++i) asm volatile("" : "+v"(q[i]));
    char* po = reinterpret_cast<char*>(static_cast<T*>(a.out) + (cnt ? lo + t.ty : lo) * a.ldo + t.tx * V);
#pragma unroll
    for (int i = 0; i < kWaveHold; ++i)
        if (i < cnt) {
            norm_store<T, ACT, COL>(reinterpret_cast<T*>(po), q[i], k, rw, a.slope, nc);
            po += so;
        }
}

// First pass, three kinds of workgroups in one launch: the first graph_blocks
// take short graphs one at a time (and give graphs without rows their
// statistics), the next wave_blocks the shortest ones, four at a time, and the
// rest the chunks' pieces of long graphs: mean and squares about it.  (With
// the wavefronts' graphs first all of them start at once and wait for memory
// and compute together: 54 us for 4096 graphs of 25 rows of 256 bf16, 45 in
// this order.)
template <class T, int ACT, bool COL>
__global__ __launch_bounds__(kThreads, COL ? 3 : 4) void norm_first(NormArgs a) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __attribute__((aligned(16))) float sh[];
    const Slots sl = slots_of<COL>(a.d, a.gd, a.tx, V);
    const int d = static_cast<int>(a.d);
    Cols<V, COL> k;
    if (blockIdx.x >= a.graph_blocks && blockIdx.x < a.graph_blocks + a.wave_blocks) {
        const Team<64> t(a, sl, 1, sh);
        k.init(a, t.tx * V);
        for (int64_t g = 4 * (static_cast<int64_t>(blockIdx.x) - a.graph_blocks) + (threadIdx.x >> 6); g < a.n_seg; g += 4 * a.wave_blocks) {
            const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
            if (lo < hi && hi - lo <= a.wave_rows) norm_held<T, ACT, COL>(a, sl, t, k, d - t.tx * V, g, lo, hi);
        }
        return;
    }
    const Team<kThreads> t(a, sl, 1, sh);
    const int nc = d - t.tx * V;
    bool ready = false;
    if (blockIdx.x < a.graph_blocks) {
        for (int64_t g = blockIdx.x; g < a.n_seg; g += a.graph_blocks) {
            const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
            if (hi <= lo) {
                for (int i = threadIdx.x; i < a.groups; i += kThreads) {
                    a.mean[g * a.groups + i] = 0.f;
                    a.rstd[g * a.groups + i] = 1.f / sqrtf(a.eps);
                }
            }
            if (hi - lo <= (a.wave_blocks ? a.wave_rows : 0) || hi - lo > a.short_rows) continue;
            if (!ready) k.init(a, t.tx * V);
            ready = true;
            const float itot = norm_stats<T, COL>(a, sl, t, k, nc, lo, hi);
            float rw[V];
            put_stats(a, t, k, g, itot, rw);
            // (every row is read before it is written, by the same thread)
            apply_rows<T, ACT, COL>(a, t, lo, hi, k, rw, nc);
        }
    } else {
        for_pieces(a, static_cast<int64_t>(blockIdx.x) - a.graph_blocks - a.wave_blocks, [&](int64_t, int64_t lo, int64_t hi, int64_t piece) {
            if (!ready) k.init(a, t.tx * V);
            ready = true;
            const float itot = norm_stats<T, COL>(a, sl, t, k, nc, lo, hi);
            for (int i = threadIdx.x; i < a.groups; i += kThreads)
                a.piece[piece * a.groups + i] = make_float2(t.gs[i] * itot, t.gs[a.groups + i]);
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
    const Team<kThreads> t(a, Slots{0, 0}, 0, nullptr);
    Cols<V, COL> k;
    bool ready = false;
    // the last chunks first: they are what the first pass left in the caches
    for_pieces(a, a.n_chunks - 1 - static_cast<int64_t>(blockIdx.x), [&](int64_t g, int64_t lo, int64_t hi, int64_t) {
        if (!ready) k.init(a, t.tx * V);
        ready = true;
        k.graph(a, g);
        float rw[V];
#pragma unroll
        for (int e = 0; e < V; ++e) rw[e] = k.rstd[k.of(e)] * k.w[e];
        apply_rows<T, ACT, COL>(a, t, lo, hi, k, rw, static_cast<int>(a.d) - t.tx * V);
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

// The thread's rows of lo .. hi - 1: dX.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void dx_rows(const NormArgs& a, const Team<kThreads>& t, int64_t lo, int64_t hi,
                                        const Cols<Vec<T>::N, COL>& k, const float (&m0)[Cols<Vec<T>::N, COL>::G],
                                        const float (&m1)[Cols<Vec<T>::N, COL>::G], int nc) {
    constexpr int64_t ES = sizeof(T);
    const uint32_t cnt = t.count(lo, hi);
    if (!cnt) return;
    const int64_t r = lo + t.ty, c0 = t.tx * Vec<T>::N;
    char* po = reinterpret_cast<char*>(static_cast<T*>(a.out) + r * a.ldo + c0);
    each_row<true>(static_cast<const T*>(a.x) + r * a.ldx + c0, t.rows * a.ldx * ES,
                   static_cast<const T*>(a.g) + r * a.ldg + c0, t.rows * a.ldg * ES, cnt, [&](u32x4_t qx, u32x4_t qg) {
                       norm_dx_store<T, ACT, COL>(reinterpret_cast<T*>(po), qx, qg, k, m0, m1, a.slope, nc);
                       po += t.rows * a.ldo * ES;
                   });
}

// Rows lo .. hi - 1 of graph g: the column sums of a and a xhat added to the
// thread's place of acc ([2][a.ty][d]), the groups' sums
// of h and h xhat (t.gs) and, for a whole graph (piece -1), dX.
template <class T, int ACT, bool COL>
__device__ __forceinline__ void norm_bwd_part(const NormArgs& a, const Slots& sl, const Team<kThreads>& t,
                                              Cols<Vec<T>::N, COL>& k, float* acc, int64_t g, int64_t lo,
                                              int64_t hi, int64_t piece) {
    constexpr int V = Vec<T>::N;
    constexpr int64_t ES = sizeof(T);
    const int d = static_cast<int>(a.d), c0 = t.tx * V, nc = d - c0;
    k.graph(a, g);
    float t0[V], t1[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t0[e] = t1[e] = 0.f;
    const uint32_t cnt = t.count(lo, hi);
    if (cnt) {
        const int64_t r = lo + t.ty;
        each_row<true>(static_cast<const T*>(a.x) + r * a.ldx + c0, t.rows * a.ldx * ES,
                       static_cast<const T*>(a.g) + r * a.ldg + c0, t.rows * a.ldg * ES, cnt, [&](u32x4_t qx, u32x4_t qg) {
                           float f[V], q[V];
                           unpack_vec<T>(qx, f);
                           unpack_vec<T>(qg, q);
#pragma unroll
                           for (int e = 0; e < V; ++e) {
                               float xh;
                               const int j = k.of(e);
                               const float u = grad_a<ACT>(f[e], q[e], k.mean[j], k.rstd[j], Affine<ACT>(k.rstd[j], k.w[e]),
                                                           k.v[e], a.slope, xh);
                               t0[e] += u;
                               t1[e] = fmaf(u, xh, t1[e]);
                           }
                       });
        float* p = acc + t.ty * d + c0;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nc) {
                p[e] += t0[e];
                p[a.ty * d + e] += t1[e];
            }
    }
    if (!a.out) return;
    float v[2][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v[0][e] = e < nc ? t0[e] * k.w[e] : 0.f;
        v[1][e] = e < nc ? t1[e] * k.w[e] : 0.f;
    }
    group_sums<2, V, COL>(a, sl, t, nc, v, t.gs);
    if (piece >= 0) {
        for (int i = t.tid; i < a.groups; i += kThreads) a.piece[piece * a.groups + i] = make_float2(t.gs[i], t.gs[a.groups + i]);
    } else {
        const float inv = 1.f / (static_cast<float>(hi - lo) * static_cast<float>(a.gd));
        float m0[Cols<V, COL>::G], m1[Cols<V, COL>::G];
#pragma unroll
        for (int e = 0; e < Cols<V, COL>::G; ++e) {
            m0[e] = t.gs[k.grp[e]] * inv;
            m1[e] = t.gs[a.groups + k.grp[e]] * inv;
        }
        dx_rows<T, ACT, COL>(a, t, lo, hi, k, m0, m1, nc);
    }
}

// First pass: dX of short graphs whole (when wanted), the pieces' sums of h
// and h xhat of long ones, and each workgroup's column sums of a and a xhat;
// workgroups as in the forward pass.
template <class T, int ACT, bool COL>
__global__ __launch_bounds__(kThreads, COL ? 2 : 3) void norm_bwd_first(NormArgs a) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __attribute__((aligned(16))) float sh[];
    const Slots sl = slots_of<COL>(a.d, a.gd, a.tx, V);
    const int d = static_cast<int>(a.d);
    float* acc = sh + 2 * a.ty * sl.n + stat_floats(a);
    for (int i = threadIdx.x; i < 2 * a.ty * d; i += kThreads) acc[i] = 0.f;
    __syncthreads();
    Cols<V, COL> k;
    const Team<kThreads> t(a, sl, 2, sh);
    k.init(a, t.tx * V);
    if (blockIdx.x < a.graph_blocks) {
        for (int64_t g = blockIdx.x; g < a.n_seg; g += a.graph_blocks) {
            const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
            if (lo < hi && hi - lo <= a.short_rows) norm_bwd_part<T, ACT, COL>(a, sl, t, k, acc, g, lo, hi, -1);
        }
    } else {
        for_pieces(a, static_cast<int64_t>(blockIdx.x) - a.graph_blocks, [&](int64_t g, int64_t lo, int64_t hi, int64_t piece) {
            norm_bwd_part<T, ACT, COL>(a, sl, t, k, acc, g, lo, hi, piece);
        });
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
    const Team<kThreads> t(a, Slots{0, 0}, 0, nullptr);
    Cols<V, COL> k;
    k.init(a, t.tx * V);
    for_pieces(a, a.n_chunks - 1 - static_cast<int64_t>(blockIdx.x), [&](int64_t g, int64_t lo, int64_t hi, int64_t) {
        k.graph(a, g);
        float m0[Cols<V, COL>::G], m1[Cols<V, COL>::G];
#pragma unroll
        for (int e = 0; e < Cols<V, COL>::G; ++e) {
            const float2 q = a.stat[g * a.groups + k.grp[e]];
            m0[e] = q.x;
            m1[e] = q.y;
        }
        dx_rows<T, ACT, COL>(a, t, lo, hi, k, m0, m1, static_cast<int>(a.d) - t.tx * V);
    });
}

struct Plan {
    int tx, ty;
    int64_t rows_per_chunk, n_chunks, max_chunks, short_rows;   // max_chunks: of up to n_rows rows
    int64_t wave_rows, graph_blocks, wave_blocks, chunk_blocks;   // of the first pass
    int64_t blocks() const { return graph_blocks + wave_blocks + chunk_blocks; }
};

// At most kMaxChunks chunks, of at least half a short graph.
Plan norm_plan(int64_t n_rows, int64_t d, int64_t n_seg, bool one, bool bwd, sag_dtype dt) {
    Plan p;
    p.tx = static_cast<int>(cdiv(d, vec_elems(dt)));
    p.ty = kThreads / p.tx;
    p.short_rows = kShort * static_cast<int64_t>(p.ty);
    p.rows_per_chunk = cdiv(n_rows, kMaxChunks);
    if (p.rows_per_chunk < p.short_rows / 2) p.rows_per_chunk = p.short_rows / 2;
    p.n_chunks = cdiv(n_rows, p.rows_per_chunk);
    p.max_chunks = cdiv(n_rows, p.short_rows / 2) < kMaxChunks ? cdiv(n_rows, p.short_rows / 2) : kMaxChunks;
    // graphs are met from their lengths on the device; the host knows that no
    // graph is long when all rows make a short one, and the length of the one
    // graph of all rows
    const bool all_short = n_rows <= p.short_rows;
    p.chunk_blocks = all_short || n_seg == 0 ? 0 : p.n_chunks;
    const bool graphs = !(one && !all_short);
    p.graph_blocks = graphs ? (n_seg < kMaxGraphBlocks ? n_seg : kMaxGraphBlocks) : 0;
    // a wavefront has two rows of threads or more there: wider rows would
    // leave up to half its lanes without a column.  A batch of few graphs
    // has workgroups to spare (25 rows of 256 bf16, 8 groups, workgroups ->
    // wavefronts: 256 graphs 16.7 -> 17.8 us, 512 20.3 -> 19.4, 4096 64 ->
    // 52; graphs of 100 rows, all past wave_rows, lose 2%: 154 -> 157).  The
    // backward pass, of two inputs, was no faster so (57 us for 1200 graphs
    // of 25 rows of 100 fp32, 54 by workgroups).
    p.wave_rows = p.tx <= 32 ? kWaveHold * static_cast<int64_t>(64 / p.tx) : 0;
    p.wave_blocks = !bwd && graphs && p.wave_rows && n_seg >= kManyGraphs ? (n_seg < 4 * kMaxGraphBlocks ? cdiv(n_seg, 4) : kMaxGraphBlocks) : 0;
    return p;
}

// The joining kernel's blocks: at most 2048 over the graphs, and with fewer
// graphs than 256 two groups each (128 parts a group).
dim3 join_grid(NormArgs& a) {
    a.seg_per_block = cdiv(a.n_seg, 2048);
    a.grp_per_block = a.n_seg < 256 && a.groups > 2 ? 2 : a.groups;
    return dim3(static_cast<unsigned>(cdiv(a.n_seg, a.seg_per_block)), static_cast<unsigned>(cdiv(a.groups, a.grp_per_block)));
}

// Lanes that add up a group's slots: what gives every group some at once, as
// many of them across the slots as a row of threads has.
void set_group_lanes(NormArgs& a, int per_group) {
    a.lanes_per_group = a.lanes_per_slots = 1;
    while (a.lanes_per_group < 64 && 2 * a.lanes_per_group * a.groups <= kThreads) a.lanes_per_group *= 2;
    while (a.lanes_per_slots < per_group && a.lanes_per_slots < 64) a.lanes_per_slots *= 2;
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
    w.piece = c.take<float2>((p.max_chunks + n_seg) * groups);
    if (bwd) {
        w.stat = c.take<float2>(n_seg * groups);
        w.col = c.take<float>((p.blocks() - p.chunk_blocks + p.max_chunks) * 2 * d);
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
    return norm_ws(norm_plan(n_rows, d, n_seg, false, false, dt), d, n_seg, groups, false, nullptr, 0).used;
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
    const Plan p = norm_plan(n_rows, d, n_seg, !seg, false, dt);
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
    a.piece = q.piece; a.rows_per_chunk = p.rows_per_chunk; a.n_chunks = p.n_chunks; a.short_rows = p.short_rows; a.wave_rows = p.wave_rows; a.graph_blocks = p.graph_blocks; a.wave_blocks = p.wave_blocks; a.tx = p.tx; a.ty = p.ty;
    const unsigned first = static_cast<unsigned>(p.blocks());
    const unsigned nc = static_cast<unsigned>(p.chunk_blocks);
    const dim3 jgrid = join_grid(a);
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto tag) {
            using T = decltype(tag);
            by_column(a.gd % Vec<T>::N != 0, [&](auto cc) {
                constexpr bool COL = decltype(cc)::value;
                const size_t lds = (static_cast<size_t>(p.ty) * slots_of<COL>(d, a.gd, p.tx, Vec<T>::N).n + stat_floats(a)) * 4;
                set_group_lanes(a, slots_of<COL>(d, a.gd, p.tx, Vec<T>::N).per_group);
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
    return norm_ws(norm_plan(n_rows, d, n_seg, false, true, dt), d, n_seg, groups, true, nullptr, 0).used;
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
    const Plan p = norm_plan(n_rows, d, n_seg, !seg, true, dt);
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
    a.rows_per_chunk = p.rows_per_chunk; a.n_chunks = p.n_chunks; a.short_rows = p.short_rows; a.wave_rows = p.wave_rows; a.graph_blocks = p.graph_blocks; a.wave_blocks = p.wave_blocks; a.tx = p.tx; a.ty = p.ty;
    const unsigned first = static_cast<unsigned>(p.blocks());
    const unsigned nc = static_cast<unsigned>(p.chunk_blocks);
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto tag) {
            using T = decltype(tag);
            if (first)
                by_column(a.gd % Vec<T>::N != 0, [&](auto cc) {
                    constexpr bool COL = decltype(cc)::value;
                    const size_t lds = (static_cast<size_t>(2 * p.ty) * (d + slots_of<COL>(d, a.gd, p.tx, Vec<T>::N).n) + stat_floats(a)) * 4;
                    set_group_lanes(a, slots_of<COL>(d, a.gd, p.tx, Vec<T>::N).per_group);
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
