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
// each, whatever the graphs' lengths; chunk c and graph g meet in at most one
// piece, and the pieces in row order are a staircase, so piece (c, g) is
// number c + g: every piece has a place of its own without a plan, and a
// graph's pieces are neighbours.  A piece's sums are joined per graph in
// piece order by a second kernel (in 64 bits), and a third pass applies them.
// The statistics are exact about a mean: each thread takes the mean of the
// few values it holds first and their squares about it, and parts are joined
// by the pairwise formula of Chan, Golub and LeVeque, so that a large mean
// does not swallow the variance.
#include <type_traits>

#include "drop.h"
#include "ops.h"
#include "trace.h"

namespace sag {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;             // rows a thread holds at once
constexpr int64_t kMaxChunks = 2048;  // eight workgroups per CU

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
    float* col;                   // backward: [n_chunks][2][d] column sums
    int64_t rows_per_chunk, n_chunks;
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

// Calls f(graph, first row, end row, piece) for each piece of this chunk, the
// same for every thread of the workgroup (all of them have to take part).
template <class F>
__device__ __forceinline__ void for_pieces(const NormArgs& a, int64_t chunk, F&& f) {
    int64_t r = chunk * a.rows_per_chunk;
    const int64_t end = r + a.rows_per_chunk < a.n_rows ? r + a.rows_per_chunk : a.n_rows;
    int64_t g = seg_of(a, r);
    if (g < 0) {                       // rows before the first graph
        g = 0;
        r = seg_at(a, 0);
    }
    while (r < end) {
        if (g >= a.n_seg) break;       // rows behind the last graph
        const int64_t ge = seg_at(a, g + 1);
        const int64_t e = ge < end ? ge : end;
        if (r < e) f(g, r, e, chunk + g);
        if (e >= end) break;
        r = e > r ? e : r;
        // the next graph with rows (empty ones share its start)
        ++g;
        if (g < a.n_seg && seg_at(a, g + 1) <= r) {
            const int64_t q = seg_of(a, r);
            g = q > g ? q : g;         // (forward only, whatever seg holds)
        }
    }
}

// Joins (n2, m2, s2) into (n, m, s): counts, means, sums of squares about the mean.
__device__ __forceinline__ void join(float& n, float& m, float& s, float n2, float m2, float s2) {
    const float t = n + n2;
    if (n2 == 0.f) return;
    const float f = n2 / t, dm = m2 - m;
    s += s2 + dm * dm * n * f;
    m += dm * f;
    n = t;
}

template <class T>
__global__ __launch_bounds__(kThreads) void norm_stats(NormArgs a) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __attribute__((aligned(16))) float sh[];
    // [ty][d] means, [ty][d] squares; then the columns' own
    const int d = static_cast<int>(a.d);
    float* sm = sh;
    float* ss = sh + a.ty * d;
    const int tx = threadIdx.x % a.tx, ty = threadIdx.x / a.tx;
    const bool on = ty < a.ty;
    const int c0 = tx * V;
    const T* x = static_cast<const T*>(a.x) + c0;
    const int nc = d - c0 < V ? d - c0 : V;
    for_pieces(a, blockIdx.x, [&](int64_t g, int64_t lo, int64_t hi, int64_t piece) {
        float n = 0.f, m[V], s[V];
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] = s[e] = 0.f;
        if (on) {
            for (int64_t r = lo + ty; r < hi; r += static_cast<int64_t>(kBatch) * a.ty) {
                uint4 q[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int64_t rk = r + static_cast<int64_t>(k) * a.ty;
                    q[k] = *reinterpret_cast<const uint4*>(x + (rk < hi ? rk : r) * a.ldx);
                }
                const int64_t left = (hi - r + a.ty - 1) / a.ty;
                const int cnt = left < kBatch ? static_cast<int>(left) : kBatch;
                const float inv = 1.f / static_cast<float>(cnt);
                float bm[V], bs[V];
#pragma unroll
                for (int e = 0; e < V; ++e) bm[e] = bs[e] = 0.f;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    float f[V];
                    unpack<T>(q[k], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) bm[e] += k < cnt ? f[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < V; ++e) bm[e] = cnt == 1 ? bm[e] : bm[e] * inv;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    float f[V];
                    unpack<T>(q[k], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float c = f[e] - bm[e];
                        bs[e] += k < cnt ? c * c : 0.f;
                    }
                }
                if (n == 0.f) {
#pragma unroll
                    for (int e = 0; e < V; ++e) { m[e] = bm[e]; s[e] = bs[e]; }
                    n = static_cast<float>(cnt);
                } else {
                    const float t = n + static_cast<float>(cnt), f = static_cast<float>(cnt) / t;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float dm = bm[e] - m[e];
                        s[e] += bs[e] + dm * dm * n * f;
                        m[e] += dm * f;
                    }
                    n = t;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < nc) {
                    sm[ty * d + c0 + e] = m[e];
                    ss[ty * d + c0 + e] = s[e];
                }
        }
        __syncthreads();
        // the row threads of each column, in order
        const int64_t len = hi - lo;
        for (int c = threadIdx.x; c < d; c += kThreads) {
            float cn = static_cast<float>((len + a.ty - 1) / a.ty), cm = sm[c], cs = ss[c];
            for (int k = 1; k < a.ty; ++k) {
                const int64_t nk = (len - k + a.ty - 1) / a.ty;
                if (k < len) join(cn, cm, cs, static_cast<float>(nk), sm[k * d + c], ss[k * d + c]);
            }
            sm[c] = cm;
            ss[c] = cs;
        }
        __syncthreads();
        // the columns of each group: lanes across the columns
        int lpg = 1;
        while (lpg < 64 && lpg < a.gd) lpg *= 2;
        const int gl = threadIdx.x % lpg;
        const float fl = static_cast<float>(len), invd = 1.f / static_cast<float>(a.gd);
        for (int gb = 0; gb < a.groups; gb += kThreads / lpg) {
            const int gi = gb + threadIdx.x / lpg;
            const bool ok = gi < a.groups;
            float sum = 0.f;
            if (ok) for (int c = gl; c < a.gd; c += lpg) sum += sm[gi * a.gd + c];
            for (int o = 1; o < lpg; o *= 2) sum += __shfl_xor(sum, o, 64);
            const float gm = a.gd == 1 ? sum : sum * invd;
            float sq = 0.f;
            if (ok) for (int c = gl; c < a.gd; c += lpg) {
                const float dm = sm[gi * a.gd + c] - gm;
                sq += ss[gi * a.gd + c] + fl * dm * dm;
            }
            for (int o = 1; o < lpg; o *= 2) sq += __shfl_xor(sq, o, 64);
            if (ok && gl == 0) a.piece[piece * a.groups + gi] = make_float2(gm, sq);
        }
        __syncthreads();
    });
}

// Joins a graph's pieces per group: blocks of 16 groups by 16 threads, each
// thread every 16th piece, then the threads in order.  BWD: the pieces hold
// sums of h and h xhat.
constexpr int kJoinG = 16, kJoinP = kThreads / kJoinG;

template <bool BWD>
__global__ __launch_bounds__(kThreads) void norm_join(NormArgs a) {
    __shared__ double p0[kThreads], p1[kThreads];
    const int64_t g = blockIdx.x;
    const int gi = blockIdx.y * kJoinG + threadIdx.x % kJoinG;
    const int part = threadIdx.x / kJoinG;
    const int64_t lo = seg_at(a, g), hi = seg_at(a, g + 1);
    const bool ok = gi < a.groups && lo < hi;
    const int64_t first = lo / a.rows_per_chunk, last = hi > lo ? (hi - 1) / a.rows_per_chunk : first - 1;
    double s0 = 0.0, s1 = 0.0, c = 0.0;
    if (ok) {
        if constexpr (!BWD) c = a.piece[(first + g) * a.groups + gi].x;
        for (int64_t k = first + part; k <= last; k += kJoinP) {
            const float2 q = a.piece[(k + g) * a.groups + gi];
            if constexpr (BWD) {
                s0 += q.x;
                s1 += q.y;
            } else {
                const int64_t b = k * a.rows_per_chunk, e = b + a.rows_per_chunk;
                const double n = static_cast<double>((e < hi ? e : hi) - (b > lo ? b : lo)) * a.gd;
                const double dm = q.x - c;
                s0 += n * dm;
                s1 += q.y + n * dm * dm;
            }
        }
    }
    p0[threadIdx.x] = s0;
    p1[threadIdx.x] = s1;
    __syncthreads();
    if (part == 0 && gi < a.groups) {
        for (int k = 1; k < kJoinP; ++k) {
            s0 += p0[k * kJoinG + threadIdx.x];
            s1 += p1[k * kJoinG + threadIdx.x];
        }
        const double n = hi > lo ? static_cast<double>(hi - lo) * a.gd : 1.0;
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
}

// This thread's columns: the affine and, per graph, the statistics.
template <int V>
struct Cols {
    float w[V], v[V], mean[V], rstd[V];
    int grp[V];
    __device__ __forceinline__ void init(const NormArgs& a, int c0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = c0 + e < a.d ? c0 + e : static_cast<int>(a.d) - 1;
            w[e] = a.w ? a.w[c] : 1.f;
            v[e] = a.v ? a.v[c] : 0.f;
            grp[e] = c / a.gd;
        }
    }
    __device__ __forceinline__ void graph(const NormArgs& a, int64_t g) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            mean[e] = a.mean[g * a.groups + grp[e]];
            rstd[e] = a.rstd[g * a.groups + grp[e]];
        }
    }
};

template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void norm_apply(NormArgs a) {
    constexpr int V = Vec<T>::N;
    const int tx = threadIdx.x % a.tx;
    // (a thread past the last row of threads walks along with no rows: the
    // search for a row's graph takes whole wavefronts)
    const int64_t ty = threadIdx.x / a.tx < a.ty ? threadIdx.x / a.tx : a.n_rows;
    const int c0 = tx * V;
    const int nc = a.d - c0 < V ? static_cast<int>(a.d) - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    T* out = static_cast<T*>(a.out) + c0;
    Cols<V> k;
    k.init(a, c0);
    for_pieces(a, blockIdx.x, [&](int64_t g, int64_t lo, int64_t hi, int64_t) {
        k.graph(a, g);
        for (int64_t r = lo + ty; r < hi; r += 4 * static_cast<int64_t>(a.ty)) {
            uint4 q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ri = r + i * static_cast<int64_t>(a.ty);
                q[i] = *reinterpret_cast<const uint4*>(x + (ri < hi ? ri : r) * a.ldx);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ri = r + i * static_cast<int64_t>(a.ty);
                if (ri >= hi) continue;
                float f[V];
                unpack<T>(q[i], f);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    f[e] = act_value<ACT>((f[e] - k.mean[e]) * k.rstd[e] * k.w[e] + k.v[e], a.slope);
                store_first<T>(out + ri * a.ldo, f, nc);
            }
        }
    });
}

// a = act'(z) g of one element, and xhat.  ReLU's and leaky ReLU's step at
// z = 0 is decided in 64 bits where fp32 cannot tell the side (|z| within
// its rounding error of about 2^-22 |v|): the gradient then has the sides of
// the formula itself, not of one rounding of it.
template <int ACT>
__device__ __forceinline__ float grad_a(float x, float g, float mean, float rstd, float w, float v, float slope,
                                        float& xhat) {
    xhat = (x - mean) * rstd;
    float z = xhat * w + v;
    if constexpr (ACT == SAG_ACT_RELU || ACT == SAG_ACT_LEAKY_RELU) {
        if (fabsf(z) <= fabsf(v) * 0x1p-20f) {
            const double zd = (static_cast<double>(x) - static_cast<double>(mean)) * static_cast<double>(rstd) *
                                  static_cast<double>(w) +
                              static_cast<double>(v);
            z = zd > 0.0 ? 1.f : (zd < 0.0 ? -1.f : 0.f);
        }
    }
    return act_grad<ACT>(z, slope) * g;
}

template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_sums(NormArgs a) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __attribute__((aligned(16))) float sh[];
    const int d = static_cast<int>(a.d);
    float* s0 = sh;                       // [ty][d]: sums of a, then a's of each column
    float* s1 = sh + a.ty * d;            // sums of a xhat
    float* acc = sh + 2 * a.ty * d;       // [2][d] of the whole chunk
    const int tx = threadIdx.x % a.tx, ty = threadIdx.x / a.tx;
    const bool on = ty < a.ty;
    const int c0 = tx * V;
    const int nc = d - c0 < V ? d - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    const T* gr = static_cast<const T*>(a.g) + c0;
    for (int c = threadIdx.x; c < 2 * d; c += kThreads) acc[c] = 0.f;
    Cols<V> k;
    if (on) k.init(a, c0);
    for_pieces(a, blockIdx.x, [&](int64_t g, int64_t lo, int64_t hi, int64_t piece) {
        if (on) {
            k.graph(a, g);
            float t0[V], t1[V];
#pragma unroll
            for (int e = 0; e < V; ++e) t0[e] = t1[e] = 0.f;
            for (int64_t r = lo + ty; r < hi; r += 4 * static_cast<int64_t>(a.ty)) {
                uint4 qx[4], qg[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t ri = r + i * static_cast<int64_t>(a.ty);
                    const int64_t rc = ri < hi ? ri : r;
                    qx[i] = *reinterpret_cast<const uint4*>(x + rc * a.ldx);
                    qg[i] = *reinterpret_cast<const uint4*>(gr + rc * a.ldg);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (r + i * static_cast<int64_t>(a.ty) >= hi) continue;
                    float f[V], q[V];
                    unpack<T>(qx[i], f);
                    unpack<T>(qg[i], q);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float xh;
                        const float t = grad_a<ACT>(f[e], q[e], k.mean[e], k.rstd[e], k.w[e], k.v[e], a.slope, xh);
                        t0[e] += t;
                        t1[e] += t * xh;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < nc) {
                    s0[ty * d + c0 + e] = t0[e];
                    s1[ty * d + c0 + e] = t1[e];
                }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += kThreads) {
            float u0 = 0.f, u1 = 0.f;
            for (int j = 0; j < a.ty; ++j) {
                u0 += s0[j * d + c];
                u1 += s1[j * d + c];
            }
            acc[c] += u0;
            acc[d + c] += u1;
            const float w = a.w ? a.w[c] : 1.f;
            s0[c] = u0 * w;
            s1[c] = u1 * w;
        }
        __syncthreads();
        int lpg = 1;
        while (lpg < 64 && lpg < a.gd) lpg *= 2;
        const int gl = threadIdx.x % lpg;
        for (int gb = 0; gb < a.groups; gb += kThreads / lpg) {
            const int gi = gb + threadIdx.x / lpg;
            const bool ok = gi < a.groups;
            float u0 = 0.f, u1 = 0.f;
            if (ok) for (int c = gl; c < a.gd; c += lpg) {
                u0 += s0[gi * a.gd + c];
                u1 += s1[gi * a.gd + c];
            }
            for (int o = 1; o < lpg; o *= 2) {
                u0 += __shfl_xor(u0, o, 64);
                u1 += __shfl_xor(u1, o, 64);
            }
            if (ok && gl == 0) a.piece[piece * a.groups + gi] = make_float2(u0, u1);
        }
        __syncthreads();
    });
    if (a.col) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * d; c += kThreads) a.col[blockIdx.x * 2 * a.d + c] = acc[c];
    }
}

// dv and dw: the chunks' column sums in chunk order, 16 columns by 16 threads.
__global__ __launch_bounds__(kThreads) void norm_cols(const float* __restrict__ col, int64_t n_chunks, int64_t d,
                                                      float* __restrict__ dw, float* __restrict__ dv) {
    __shared__ double p[kThreads];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x % 16;   // of 2 d: sums of a, then of a xhat
    const int part = threadIdx.x / 16;
    double s = 0.0;
    if (c < 2 * d)
        for (int64_t k = part; k < n_chunks; k += 16) s += col[k * 2 * d + c];
    p[threadIdx.x] = s;
    __syncthreads();
    if (part == 0 && c < 2 * d) {
        for (int k = 1; k < 16; ++k) s += p[k * 16 + threadIdx.x];
        if (c < d) { if (dv) dv[c] = static_cast<float>(s); }
        else if (dw) dw[c - d] = static_cast<float>(s);
    }
}

template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_apply(NormArgs a) {
    constexpr int V = Vec<T>::N;
    const int tx = threadIdx.x % a.tx;
    // (a thread past the last row of threads walks along with no rows: the
    // search for a row's graph takes whole wavefronts)
    const int64_t ty = threadIdx.x / a.tx < a.ty ? threadIdx.x / a.tx : a.n_rows;
    const int c0 = tx * V;
    const int nc = a.d - c0 < V ? static_cast<int>(a.d) - c0 : V;
    const T* x = static_cast<const T*>(a.x) + c0;
    const T* gr = static_cast<const T*>(a.g) + c0;
    T* out = static_cast<T*>(a.out) + c0;
    Cols<V> k;
    k.init(a, c0);
    for_pieces(a, blockIdx.x, [&](int64_t g, int64_t lo, int64_t hi, int64_t) {
        k.graph(a, g);
        float m0[V], m1[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 q = a.stat[g * a.groups + k.grp[e]];
            m0[e] = q.x;
            m1[e] = q.y;
        }
        for (int64_t r = lo + ty; r < hi; r += 4 * static_cast<int64_t>(a.ty)) {
            uint4 qx[4], qg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ri = r + i * static_cast<int64_t>(a.ty);
                const int64_t rc = ri < hi ? ri : r;
                qx[i] = *reinterpret_cast<const uint4*>(x + rc * a.ldx);
                qg[i] = *reinterpret_cast<const uint4*>(gr + rc * a.ldg);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ri = r + i * static_cast<int64_t>(a.ty);
                if (ri >= hi) continue;
                float f[V], q[V];
                unpack<T>(qx[i], f);
                unpack<T>(qg[i], q);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float xh;
                    const float t = grad_a<ACT>(f[e], q[e], k.mean[e], k.rstd[e], k.w[e], k.v[e], a.slope, xh);
                    f[e] = k.rstd[e] * (t * k.w[e] - m0[e] - xh * m1[e]);
                }
                store_first<T>(out + ri * a.ldo, f, nc);
            }
        }
    });
}

struct Plan {
    int tx, ty;
    int64_t rows_per_chunk, n_chunks;
};

// At most kMaxChunks chunks of at least 4 rows a thread row.
Plan norm_plan(int64_t n_rows, int64_t d, sag_dtype dt) {
    Plan p;
    p.tx = static_cast<int>(cdiv(d, vec_elems(dt)));
    p.ty = kThreads / p.tx;
    const int64_t least = 4 * p.ty;
    p.rows_per_chunk = cdiv(n_rows > 0 ? n_rows : 1, kMaxChunks);
    if (p.rows_per_chunk < least) p.rows_per_chunk = least;
    p.n_chunks = cdiv(n_rows, p.rows_per_chunk);
    return p;
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
        w.col = c.take<float>(p.n_chunks * 2 * d);
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
    return norm_ws(norm_plan(n_rows, d, dt), d, n_seg, groups, false, nullptr, 0).used;
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
    const Plan p = norm_plan(n_rows, d, dt);
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
    a.piece = q.piece; a.rows_per_chunk = p.rows_per_chunk; a.n_chunks = p.n_chunks; a.tx = p.tx; a.ty = p.ty;
    const size_t lds = static_cast<size_t>(2 * p.ty) * d * 4;
    const unsigned nc = static_cast<unsigned>(p.n_chunks);
    const dim3 jgrid(static_cast<unsigned>(n_seg), static_cast<unsigned>(cdiv(groups, kJoinG)));
    auto go = [&](auto tag) {
        using T = decltype(tag);
        if (nc) norm_stats<T><<<nc, kThreads, lds, s>>>(a);
        norm_join<false><<<jgrid, kThreads, 0, s>>>(a);
        if (nc) with_act(act, [&](auto ac) { norm_apply<T, decltype(ac)::value><<<nc, kThreads, 0, s>>>(a); });
    };
    if (dt == SAG_BF16) go(uint16_t{});
    else go(float{});
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

extern "C" size_t sag_group_norm_backward_workspace_bytes(int64_t n_rows, int64_t d, int64_t groups, int64_t n_seg,
                                                          sag_dtype dt) {
    if (n_rows < 0 || d < 1 || groups < 1 || n_seg < 0 || (dt != SAG_F32 && dt != SAG_BF16) || d > 256 * vec_elems(dt)) return 0;
    return norm_ws(norm_plan(n_rows, d, dt), d, n_seg, groups, true, nullptr, 0).used;
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
    const Plan p = norm_plan(n_rows, d, dt);
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
    a.rows_per_chunk = p.rows_per_chunk; a.n_chunks = p.n_chunks; a.tx = p.tx; a.ty = p.ty;
    const size_t lds = static_cast<size_t>(2 * p.ty + 2) * d * 4;
    const unsigned nc = n_seg ? static_cast<unsigned>(p.n_chunks) : 0u;
    const dim3 jgrid(static_cast<unsigned>(n_seg), static_cast<unsigned>(cdiv(groups, kJoinG)));
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto tag) {
            using T = decltype(tag);
            if (nc) norm_bwd_sums<T, ACT><<<nc, kThreads, lds, s>>>(a);
            if (dw || db)
                norm_cols<<<static_cast<unsigned>(cdiv(2 * d, 16)), kThreads, 0, s>>>(q.col, nc, d, dw, db);
            if (dX && nc) {
                norm_join<true><<<jgrid, kThreads, 0, s>>>(a);
                norm_bwd_apply<T, ACT><<<nc, kThreads, 0, s>>>(a);
            }
        };
        if (dt == SAG_BF16) go(uint16_t{});
        else go(float{});
    });
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}
