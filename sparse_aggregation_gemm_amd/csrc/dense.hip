// The dense layer and its gradients:
//   Z = X W + b;  Out = R + dropout(act(Z))
//   dZ = act'(Z) dropout(G);  dX = dZ W^T;  dW = X^T dZ;  db = column sums of dZ.
//
// dense_nn computes C = A B tile by tile: 128 rows by BN columns a workgroup,
// 128 bytes of k at a time through LDS (next piece in registers while the
// current one feeds the matrix cores), bf16 on v_mfma_f32_32x32x16_bf16 and
// fp32 on v_mfma_f32_32x32x2f32, sums in fp32.  The wavefronts multiply
// transposed blocks (B first, A second), so a lane holds four consecutive
// columns of one row; the sums go through LDS once more, in fp32, into lanes
// of eight consecutive columns: one generator block, one 16-byte vector of
// R, Z and Out each, and whole 128-byte lines of a row per eight lanes.
// B (the weight, or its transpose) is packed first into [N, K] with K
// contiguous and zeros up to whole tiles, so only A needs bounds.
#include <type_traits>

#include "drop.h"
#include "ops.h"
#include "trace.h"

namespace sag {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
// (a vector type, not the uint4 class, whose conditional copies go through
// private memory)
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kBM = 128;
constexpr int kRowB = 128;                 // bytes of k per tile row
constexpr int kStagePitch = 64 * 4 + 16;   // fp32 row of 64 columns, shifted 4 banks a row

// 16-byte unit u of tile row r sits at u ^ swz(r): fragment reads (32 rows,
// one unit) and row writes both spread over the banks.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

__device__ __forceinline__ int64_t xcd_tile(int64_t bid, int64_t total) {
    constexpr int64_t X = 8;
    const int64_t per = total / X, rem = total % X;
    const int64_t xcd = bid % X, local = bid / X;
    return (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + local;
}

// Zeroes elements >= n of a vector of T.
template <class T>
__device__ __forceinline__ u32x4_t keep_first(u32x4_t v, int n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) v[e] = e < n ? v[e] : 0u;
        else v[e] = 2 * e + 1 < n ? v[e] : (2 * e < n ? v[e] & 0xffffu : 0u);
    }
    return v;
}
__device__ __forceinline__ u32x4_t load16(const void* p) { return *reinterpret_cast<const u32x4_t*>(p); }
__device__ __forceinline__ void store16(void* p, u32x4_t v) { *reinterpret_cast<u32x4_t*>(p) = v; }
__device__ __forceinline__ uint4 as_uint4(u32x4_t v) { return make_uint4(v[0], v[1], v[2], v[3]); }

// Eight consecutive elements of a row: loads (columns past n read as they
// are: the pitch covers the last vector, a vector past it is not read),
// values and stores.
template <class T>
struct Eight {
    u32x4_t v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p, int live) {
        v[0] = load16(p);
        if constexpr (sizeof(T) == 4) {
            v[1] = u32x4_t{0u, 0u, 0u, 0u};
            if (live > 4) v[1] = load16(p + 4);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        unpack<T>(as_uint4(v[0]), f);
        if constexpr (sizeof(T) == 4) unpack<T>(as_uint4(v[1]), f + 4);
    }
    static __device__ __forceinline__ void put(T* p, const float (&f)[8], int live) {
        if constexpr (sizeof(T) == 2) {
            store_first<T>(p, f, live);
        } else {
            store_first<T>(p, f, live);
            if (live > 4) store_first<T>(p + 4, f + 4, live - 4);
        }
    }
};

template <class T>
struct NnArgs {
    const T* a;
    int64_t lda, M, K;
    const T* bp;          // packed B: [n_blk * BN, Kt]
    int64_t Kt, N;
    int64_t n_blk, m_blk;
    const float* bias;    // nullable
    float slope;
    DropArgs drop;
    const T* res;         // nullable
    int64_t ldr;
    T* z;                 // nullable
    int64_t ldz;
    T* out;
    int64_t ldo;
};

// WM x WN wavefronts, each MB x NB blocks of 32 x 32.
template <class T, int BN, int ACT, bool DROP>
__global__ __launch_bounds__(kThreads) void dense_nn(NnArgs<T> p) {
    constexpr int V = Vec<T>::N;
    constexpr int CK = kRowB / static_cast<int>(sizeof(T));
    constexpr int WN = BN == 128 ? 2 : 1, WM = 4 / WN;
    constexpr int MB = kBM / WM / 32, NB = BN / WN / 32;
    constexpr int UA = kBM * 8 / kThreads, UB = BN * 8 / kThreads;   // 16-byte units per thread
    constexpr int kTiles = (kBM + BN) * kRowB;
    constexpr int kStage = 4 * 32 * kStagePitch;
    __shared__ __attribute__((aligned(16))) unsigned char lds[kTiles > kStage ? kTiles : kStage];
    unsigned char* As = lds;
    unsigned char* Bs = lds + kBM * kRowB;

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const int h = lane >> 5, l32 = lane & 31;
    const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t m0 = tile / p.n_blk * kBM, n0 = tile % p.n_blk * BN;

    u32x4_t ra[UA], rb[UB];
    const int64_t last = (p.K + V - 1) / V * V - V;
    auto load = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const int q = t + i * kThreads, r = q >> 3, u = q & 7;
            const int64_t row = m0 + r < p.M ? m0 + r : p.M - 1;
            const int64_t k = k0 + u * V;
            ra[i] = load16(p.a + row * p.lda + (k < last ? k : last));
        }
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int q = t + i * kThreads, r = q >> 3, u = q & 7;
            rb[i] = load16(p.bp + (n0 + r) * p.Kt + k0 + u * V);
        }
    };
    auto store = [&](int64_t k0) {
        const bool edge = k0 + CK > p.K;
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const int q = t + i * kThreads, r = q >> 3, u = q & 7;
            const int64_t left = p.K - k0 - u * V;
            store16(As + r * kRowB + ((u ^ swz(r)) << 4),
                    edge ? keep_first<T>(ra[i], left < V ? (left > 0 ? static_cast<int>(left) : 0) : V) : ra[i]);
        }
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int q = t + i * kThreads, r = q >> 3, u = q & 7;
            store16(Bs + r * kRowB + ((u ^ swz(r)) << 4), rb[i]);
        }
    };
    f32x16_t acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    load(0);
    for (int64_t k0 = 0; k0 < p.Kt; k0 += CK) {
        store(k0);
        __syncthreads();
        if (k0 + CK < p.Kt) load(k0 + CK);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            u32x4_t a[MB], b[NB];
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int r = (wm * MB + i) * 32 + l32;
                a[i] = load16(As + r * kRowB + (((2 * s + h) ^ swz(r)) << 4));
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int r = (wn * NB + j) * 32 + l32;
                b[j] = load16(Bs + r * kRowB + (((2 * s + h) ^ swz(r)) << 4));
            }
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    if constexpr (sizeof(T) == 2) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b[j]),
                                                                             __builtin_bit_cast(bf16x8_t, a[i]),
                                                                             acc[i][j], 0, 0, 0);
                    } else {
                        // unit h holds k 4h .. 4h + 3 of the step: product q pairs k q with k 4 + q
                        const f32x4_t bb = __builtin_bit_cast(f32x4_t, b[j]);
                        const f32x4_t aa = __builtin_bit_cast(f32x4_t, a[i]);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(bb[q], aa[q], acc[i][j], 0, 0, 0);
                    }
                }
        }
        __syncthreads();
    }

    // ---- epilogue: 32 rows at a time through this wavefront's part of LDS
    unsigned char* st = lds + wave * 32 * kStagePitch;
    constexpr int UPR = NB * 4;                   // units of eight columns per row
    constexpr int RPI = 64 / UPR;                 // rows per pass over the lanes
    const int rr = lane / UPR, u = lane % UPR;
    const int64_t col = n0 + wn * NB * 32 + u * 8;
    const int live = p.N - col < 8 ? static_cast<int>(p.N - col) : 8;   // <= 0: past the columns
    float bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = p.bias && e < live ? p.bias[col + e] : 0.f;
    uint32_t call = 0;
    if constexpr (DROP) call = p.drop.call_now();
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int64_t row0 = m0 + (wm * MB + i) * 32;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<float4*>(st + l32 * kStagePitch + (j * 32 + 8 * q + 4 * h) * 4) =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int w = 0; w < 32 / RPI; ++w) {
            const int r = w * RPI + rr;
            const int64_t row = row0 + r;
            if (row >= p.M || live <= 0) continue;
            Eight<T> rv;
            if (p.res) rv.load(p.res + row * p.ldr + col, live);
            const float4 lo = *reinterpret_cast<const float4*>(st + r * kStagePitch + u * 32);
            const float4 hi = *reinterpret_cast<const float4*>(st + r * kStagePitch + u * 32 + 16);
            float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += bias[e];
            if (p.z) Eight<T>::put(p.z + row * p.ldz + col, y, live);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = act_value<ACT, T>(y[e], p.slope);
            if constexpr (DROP) {
                uint32_t dw[4];
                p.drop.draws(p.drop.node_of(row), static_cast<uint32_t>(col >> 3), call, dw);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = p.drop.apply(y[e], dw, e);
            }
            if (p.res) {
                float f[8];
                rv.get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += f[e];
            }
            Eight<T>::put(p.out + row * p.ldo + col, y, live);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Bp[n, k] = B element (k, n) at b[k * sk + n * sn], zero past K and N.
template <class T>
__global__ void dense_pack(const T* __restrict__ b, int64_t sk, int64_t sn, int64_t K, int64_t N, int64_t Kt,
                           int64_t total, T* __restrict__ bp) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const int64_t n = i / Kt, k = i % Kt;
    bp[i] = k < K && n < N ? b[k * sk + n * sn] : from_f32<T>(0.f);
}

// ---- dZ -------------------------------------------------------------------------------
// hi = dZ rounded to T; lo (bf16 only, nullable) = dZ - hi rounded: together
// the two carry 16 bits of dZ into the fp32 weight gradient.
template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void dense_dz(int64_t M, int64_t N, int64_t upr, const T* __restrict__ z,
                                                     int64_t ldz, const T* __restrict__ g, int64_t ldg, float slope,
                                                     DropArgs drop, T* __restrict__ hi, T* __restrict__ lo,
                                                     int64_t ldh) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t row = i / upr, u = i - row * upr, col = 8 * u;
    if (row >= M) return;
    const int live = N - col < 8 ? static_cast<int>(N - col) : 8;
    Eight<T> gv, zv;
    gv.load(g + row * ldg + col, live);
    if constexpr (ACT != SAG_ACT_NONE) zv.load(z + row * ldz + col, live);
    float f[8];
    gv.get(f);
    if (drop.T) {
        uint32_t dw[4];
        drop.draws(drop.node_of(row), static_cast<uint32_t>(u), drop.call_now(), dw);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = drop.apply(f[e], dw, e);
    }
    if constexpr (ACT != SAG_ACT_NONE) {
        float zf[8];
        zv.get(zf);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= act_grad<ACT>(zf[e], slope);
    }
    Eight<T>::put(hi + row * ldh + col, f, live);
    if (lo) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = f[e] - to_f32(from_f32<T>(f[e]));
        Eight<T>::put(lo + row * ldh + col, r, live);
    }
}

__global__ void add_in_place(float* __restrict__ c, const float* __restrict__ d, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) c[i] += d[i];
}

int64_t k_pad(int64_t K, sag_dtype dt) { return round_up(K, kRowB / elt_size(dt)); }
size_t pack_bytes(int64_t K, int64_t N, sag_dtype dt) {
    return static_cast<size_t>(round_up(N, 128) * k_pad(K, dt) * elt_size(dt));
}

// Packs B ([K, N]; element (k, n) at b[k sk + n sn]) and multiplies.
template <class T>
sag_status nn_run(const char* what, sag_act act, NnArgs<T> p, const T* b, int64_t sk, int64_t sn, T* bp, sag_dtype dt,
                  hipStream_t s) {
    const int BN = p.N <= 64 ? 64 : 128;
    p.Kt = k_pad(p.K, dt);
    p.bp = bp;
    p.n_blk = cdiv(p.N, BN);
    p.m_blk = cdiv(p.M, kBM);
    if (p.n_blk * p.m_blk >= (1 << 24)) return fail(SAG_E_UNSUPPORTED, std::string(what) + ": too many tiles for one launch");
    const int64_t total = p.n_blk * BN * p.Kt;
    dense_pack<T><<<dim3(static_cast<unsigned>(cdiv(total, 256))), 256, 0, s>>>(b, sk, sn, p.K, p.N, p.Kt, total, bp);
    SAG_LAUNCH_CHECK();
    TraceScope trace(trace_enabled() ? shape_name(what, dt == SAG_BF16 ? "bf16" : "f32", p.M, p.K, p.N) : std::string(),
                     s, elt_size(dt) * (p.M * p.K + p.K * p.N + p.M * p.N * (1 + (p.z ? 1 : 0) + (p.res ? 1 : 0))),
                     2 * p.M * p.K * p.N);
    const dim3 grid(static_cast<unsigned>(p.n_blk * p.m_blk));
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        if (BN == 64) {
            if (p.drop.T) dense_nn<T, 64, ACT, true><<<grid, kThreads, 0, s>>>(p);
            else dense_nn<T, 64, ACT, false><<<grid, kThreads, 0, s>>>(p);
        } else {
            if (p.drop.T) dense_nn<T, 128, ACT, true><<<grid, kThreads, 0, s>>>(p);
            else dense_nn<T, 128, ACT, false><<<grid, kThreads, 0, s>>>(p);
        }
    });
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

template <class T>
sag_status forward_typed(NnArgs<T> p, const void* W, sag_act act, sag_dtype dt, void* ws, hipStream_t s) {
    return nn_run<T>("dense", act, p, static_cast<const T*>(W), p.N, 1, static_cast<T*>(ws), dt, s);
}

struct BwdWs {
    void *bp, *hi, *lo, *tn;
    float *c2, *cs2;
    size_t tn_bytes;
    size_t used;
    bool fits;
};

BwdWs bwd_ws(int64_t M, int64_t K, int64_t N, sag_dtype dt, void* ws, size_t bytes) {
    Carver c(ws, bytes);
    BwdWs w{};
    w.bp = c.take<char>(pack_bytes(N, K, dt));
    w.hi = c.take<char>(dense_bytes(M, N, dt));
    if (dt == SAG_BF16) {
        w.lo = c.take<char>(dense_bytes(M, N, dt));
        w.c2 = c.take<float>(K * N + N);
        w.cs2 = w.c2 ? w.c2 + K * N : nullptr;
    }
    w.tn_bytes = gemm_tn_ws_bytes(M, round_up(K, vec_elems(dt)), N, dt);
    w.tn = c.take<char>(w.tn_bytes);
    w.used = c.used();
    w.fits = c.fits();
    return w;
}

template <class T>
sag_status backward_typed(int64_t M, const T* X, int64_t ldx, int64_t K, const T* W, int64_t N, sag_act act, float slope,
                          const DropArgs& drop, const T* Z, int64_t ldz, const T* G, int64_t ldg, float* dW, float* db,
                          T* dX, int64_t ldd, sag_dtype dt, const BwdWs& w, hipStream_t s) {
    const int64_t ldh = ldv(N, dt), upr = cdiv(N, 8);
    T* hi = static_cast<T*>(w.hi);
    T* lo = static_cast<T*>(w.lo);
    if (M > 0) {
        const int64_t blocks = cdiv(M * upr, kThreads);
        if (blocks >= (1 << 24)) return fail(SAG_E_UNSUPPORTED, "dense backward: too many elements for one launch");
        TraceScope trace(trace_enabled() ? shape_name("dense_dz", dt == SAG_BF16 ? "bf16" : "f32", M, N, 0) : std::string(),
                         s, elt_size(dt) * M * N * (2 + (act != SAG_ACT_NONE ? 1 : 0) + (lo ? 1 : 0)), 0);
        with_act(act, [&](auto ac) {
            dense_dz<T, decltype(ac)::value><<<dim3(static_cast<unsigned>(blocks)), kThreads, 0, s>>>(
                M, N, upr, Z, ldz, G, ldg, slope, drop, hi, lo, ldh);
        });
        SAG_LAUNCH_CHECK();
    }
    if (dX && M > 0) {
        NnArgs<T> p{};
        p.a = hi; p.lda = ldh; p.M = M; p.K = N; p.N = K;
        p.drop = DropArgs{};
        p.out = dX; p.ldo = ldd;
        SAG_TRY(nn_run<T>("dense_dx", SAG_ACT_NONE, p, W, 1, N, static_cast<T*>(w.bp), dt, s));
    }
    if (dW || db) {
        GemmA a;
        a.a1 = X; a.lda1 = ldx; a.k1 = K; a.m1 = M;
        float* cw = dW ? dW : w.c2;
        SAG_TRY(gemm_tn_run(M, N, a, hi, ldh, nullptr, 0, cw, N, db, dt, w.tn, w.tn_bytes, s));
        if (lo) {
            SAG_TRY(gemm_tn_run(M, N, a, lo, ldh, nullptr, 0, w.c2, N, db ? w.cs2 : nullptr, dt, w.tn, w.tn_bytes, s));
            if (dW) add_in_place<<<dim3(static_cast<unsigned>(cdiv(K * N, 256))), 256, 0, s>>>(dW, w.c2, K * N);
            if (db) add_in_place<<<dim3(static_cast<unsigned>(cdiv(N, 256))), 256, 0, s>>>(db, w.cs2, N);
            SAG_LAUNCH_CHECK();
        }
    }
    return SAG_OK;
}

sag_status check_sizes(const char* who, int64_t M, int64_t K, int64_t N, sag_act act, float slope, sag_dtype dt) {
    if (dt != SAG_F32 && dt != SAG_BF16) return fail(SAG_E_INVALID, std::string(who) + ": bad dtype");
    if (M < 0 || K < 1 || N < 1) return fail(SAG_E_INVALID, std::string(who) + ": bad size");
    if (K > (int64_t{1} << 24) || N > (int64_t{1} << 24)) return fail(SAG_E_UNSUPPORTED, std::string(who) + ": width above 2^24");
    if (!act_ok(act)) return fail(SAG_E_INVALID, std::string(who) + ": unknown activation");
    if (!std::isfinite(slope)) return fail(SAG_E_INVALID, std::string(who) + ": slope not finite");
    return SAG_OK;
}

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" size_t sag_dense_forward_workspace_bytes(int64_t M, int64_t K, int64_t N, sag_dtype dt) {
    (void)M;
    if (K < 1 || N < 1 || (dt != SAG_F32 && dt != SAG_BF16)) return 0;
    return pack_bytes(K, N, dt);
}

extern "C" sag_status sag_dense_layer_forward(int64_t M, const void* X, int64_t ldx, int64_t K, const void* W,
                                              const float* b, int64_t N, sag_act act, float slope,
                                              const sag_drop* drop, const void* R, int64_t ldr, sag_dtype dt, void* Z,
                                              int64_t ldz, void* Out, int64_t ldo, void* ws, size_t ws_bytes,
                                              void* stream) {
    SAG_TRY(check_sizes("dense forward", M, K, N, act, slope, dt));
    SAG_TRY(check_dense("dense X", X, M, K, ldx, dt));
    if (!W) return fail(SAG_E_INVALID, "dense forward: null W");
    if (R) SAG_TRY(check_dense("dense R", R, M, N, ldr, dt));
    if (Z) SAG_TRY(check_dense("dense Z", Z, M, N, ldz, dt));
    SAG_TRY(check_dense("dense Out", Out, M, N, ldo, dt));
    DropArgs da;
    SAG_TRY(make_drop("dense forward", drop, M, &da));
    if (M == 0) return SAG_OK;
    if (!ws || !aligned16(ws) || ws_bytes < sag_dense_forward_workspace_bytes(M, K, N, dt))
        return fail(SAG_E_WORKSPACE, "dense forward: workspace too small");
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        NnArgs<T> p{};
        p.a = static_cast<const T*>(X); p.lda = ldx; p.M = M; p.K = K; p.N = N;
        p.bias = b; p.slope = slope; p.drop = da;
        p.res = static_cast<const T*>(R); p.ldr = ldr;
        p.z = static_cast<T*>(Z); p.ldz = ldz;
        p.out = static_cast<T*>(Out); p.ldo = ldo;
        return forward_typed<T>(p, W, act, dt, ws, s);
    };
    return dt == SAG_BF16 ? go(uint16_t{}) : go(float{});
}

extern "C" size_t sag_dense_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, sag_dtype dt) {
    if (M < 0 || K < 1 || N < 1 || (dt != SAG_F32 && dt != SAG_BF16)) return 0;
    return bwd_ws(M, K, N, dt, nullptr, 0).used;
}

extern "C" sag_status sag_dense_layer_backward(int64_t M, const void* X, int64_t ldx, int64_t K, const void* W,
                                               int64_t N, sag_act act, float slope, const sag_drop* drop,
                                               const void* Z, int64_t ldz, const void* G, int64_t ldg, float* dW,
                                               float* db, void* dX, int64_t ldd, sag_dtype dt, void* ws,
                                               size_t ws_bytes, void* stream) {
    SAG_TRY(check_sizes("dense backward", M, K, N, act, slope, dt));
    if (dW || db) SAG_TRY(check_dense("dense X", X, M, K, ldx, dt));
    if (dX && !W) return fail(SAG_E_INVALID, "dense backward: null W");
    if (act != SAG_ACT_NONE) SAG_TRY(check_dense("dense Z", Z, M, N, ldz, dt));
    SAG_TRY(check_dense("dense G", G, M, N, ldg, dt));
    if (dX) SAG_TRY(check_dense("dense dX", dX, M, K, ldd, dt));
    DropArgs da;
    SAG_TRY(make_drop("dense backward", drop, M, &da));
    if (!ws || !aligned16(ws)) return fail(SAG_E_WORKSPACE, "dense backward: workspace too small");
    const BwdWs w = bwd_ws(M, K, N, dt, ws, ws_bytes);
    if (!w.fits) return fail(SAG_E_WORKSPACE, "dense backward: workspace too small");
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        return backward_typed<T>(M, static_cast<const T*>(X), ldx, K, static_cast<const T*>(W), N, act, slope, da,
                                 static_cast<const T*>(Z), ldz, static_cast<const T*>(G), ldg, dW, db,
                                 static_cast<T*>(dX), ldd, dt, w, s);
    };
    return dt == SAG_BF16 ? go(uint16_t{}) : go(float{});
}
