// Dropout over rows of dense matrices from the counter-based generator:
//   Out[r, j] = keep(r, j) ? s X[r, j] : 0  (+ addend[r, j]),
// the mask recomputed wherever it is needed (the gradient is the same call on
// the upstream gradient).  Bound: HBM (one read, one write, one more read
// with an addend); the generator's work, one block per eight elements, runs
// under the loads.
//
// A workgroup handles kUnits consecutive units of eight elements (one 16-byte
// bf16 vector or two fp32 vectors), numbered row by row, so that any width
// fills the lanes; the unit's row comes from one 64-bit division per
// workgroup and a multiply-high per unit.
#include <type_traits>

#include "drop.h"
#include "trace.h"

namespace sag {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;
constexpr int kUnits = kThreads * kPerThread;

struct Args {
    const void* x;
    int64_t ldx;
    const void* add;
    int64_t ld_add;
    void* out;
    int64_t ldo;
    int64_t n, d, upr;   // upr: units per row
    int64_t total;       // n * upr
    uint32_t magic;      // ceil(2^32 / upr): offset / upr for the small offsets below
    DropArgs drop;
};

// Eight elements from column j0 (elements past d: unspecified; a second fp32
// vector that starts at or past d is not read).
template <class T>
__device__ __forceinline__ void load_unit(const T* p, int64_t j0, int64_t d, uint4 (&v)[sizeof(T) / 2]) {
    v[0] = *reinterpret_cast<const uint4*>(p + j0);
    if constexpr (sizeof(T) == 4)
        v[1] = j0 + 4 < d ? *reinterpret_cast<const uint4*>(p + j0 + 4) : make_uint4(0, 0, 0, 0);
}

template <class T>
__device__ __forceinline__ void unpack_unit(const uint4 (&v)[sizeof(T) / 2], float (&f)[8]) {
    unpack<T>(v[0], f);
    if constexpr (sizeof(T) == 4) unpack<T>(v[1], f + 4);
}

template <class T, bool ADD>
__global__ __launch_bounds__(kThreads) void dropout_rows(Args a) {
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kUnits;
    const int64_t row_b = base / a.upr;
    const uint32_t off_b = static_cast<uint32_t>(base - row_b * a.upr);
    const uint32_t upr = static_cast<uint32_t>(a.upr);
    const uint32_t call = a.drop.call_now();
    uint4 xv[kPerThread][sizeof(T) / 2], av[ADD ? kPerThread : 1][sizeof(T) / 2];
    int64_t row[kPerThread];
    uint32_t g[kPerThread];
    uint32_t node[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        // o < upr + kUnits: in rows of kUnits units or more it is this row
        // or the next, below that o * upr < 2^32 keeps the multiply-high exact
        const uint32_t o = off_b + threadIdx.x + i * kThreads;
        const uint32_t q = upr >= kUnits ? (o >= upr ? 1u : 0u) : (upr == 1 ? o : __umulhi(o, a.magic));
        row[i] = row_b + q;
        g[i] = o - q * upr;
        const bool in = base + threadIdx.x + i * kThreads < a.total;
        if (!in) { row[i] = a.n - 1; g[i] = 0; }
        load_unit<T>(static_cast<const T*>(a.x) + row[i] * a.ldx, 8 * static_cast<int64_t>(g[i]), a.d, xv[i]);
        if constexpr (ADD)
            load_unit<T>(static_cast<const T*>(a.add) + row[i] * a.ld_add, 8 * static_cast<int64_t>(g[i]), a.d, av[i]);
        node[i] = a.drop.node_of(row[i]);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (base + threadIdx.x + i * kThreads >= a.total) continue;
        float f[8];
        unpack_unit<T>(xv[i], f);
        if (a.drop.T) {
            uint32_t w[4];
            a.drop.draws(node[i], g[i], call, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = a.drop.apply(f[e], w, e);
        }
        if constexpr (ADD) {
            float h[8];
            unpack_unit<T>(av[i], h);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += h[e];
        }
        const int64_t j0 = 8 * static_cast<int64_t>(g[i]);
        const int live = static_cast<int>(a.d - j0 < 8 ? a.d - j0 : 8);
        T* p = static_cast<T*>(a.out) + row[i] * a.ldo + j0;
        if constexpr (sizeof(T) == 2) {
            store_first<T>(p, f, live);
        } else {
            store_first<T>(p, f, live);
            if (live > 4) store_first<T>(p + 4, f + 4, live - 4);
        }
    }
}

}  // namespace
}  // namespace sag

extern "C" sag_status sag_dropout(const void* X, int64_t ldx, int64_t n, int64_t d, sag_dtype dt,
                                  const sag_drop* drop, const void* addend, int64_t ld_add, void* Out,
                                  int64_t ldo, void* stream) {
    using namespace sag;
    if (dt != SAG_F32 && dt != SAG_BF16) return fail(SAG_E_INVALID, "dropout: bad dtype");
    if (!drop) return fail(SAG_E_INVALID, "dropout: null description");
    SAG_TRY(check_dense("dropout X", X, n, d, ldx, dt));
    if (addend) SAG_TRY(check_dense("dropout addend", addend, n, d, ld_add, dt));
    SAG_TRY(check_dense("dropout Out", Out, n, d, ldo, dt));
    Args a{};
    SAG_TRY(make_drop("dropout", drop, n, &a.drop));
    if (n == 0 || d == 0) return SAG_OK;
    if (d > (int64_t{1} << 31)) return fail(SAG_E_UNSUPPORTED, "dropout: rows wider than 2^31 elements");
    a.x = X; a.ldx = ldx; a.add = addend; a.ld_add = ld_add; a.out = Out; a.ldo = ldo;
    a.n = n; a.d = d; a.upr = cdiv(d, 8);
    a.total = n * a.upr;
    a.magic = a.upr > 1 ? static_cast<uint32_t>(((uint64_t{1} << 32) + a.upr - 1) / a.upr) : 0u;
    const int64_t blocks = cdiv(a.total, kUnits);
    if (blocks >= (1 << 24)) return fail(SAG_E_UNSUPPORTED, "dropout: more units than one launch holds");
    hipStream_t s = static_cast<hipStream_t>(stream);
    TraceScope trace(trace_enabled() ? shape_name("dropout", dt == SAG_BF16 ? "bf16" : "f32", n, d, addend ? 1 : 0)
                                     : std::string(),
                     s, n * (elt_size(dt) * d * (addend ? 3 : 2) + (a.drop.nodes ? 4 : 0)), 0);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (dt == SAG_BF16) {
        if (addend) dropout_rows<uint16_t, true><<<grid, kThreads, 0, s>>>(a);
        else dropout_rows<uint16_t, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (addend) dropout_rows<float, true><<<grid, kThreads, 0, s>>>(a);
        else dropout_rows<float, false><<<grid, kThreads, 0, s>>>(a);
    }
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}
