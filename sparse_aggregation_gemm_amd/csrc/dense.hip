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
// contiguous and zeros up to whole tiles, so only A needs bounds.  Products of
// few tiles run in dense_few, the weight gradients in dense_tn (bf16) and
// dense_tn32 (fp32).  2.45M x 256 -> 256 bf16 with GELU, dropout, residual and
// Z: 1.19 ms forward (4.2 TB/s), 2.05 ms backward.
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

// The derivative of GELU and SiLU at a bf16 argument, from a table in LDS:
// act'(z) - 1/2 is odd, so act'(z) = 1/2 + z r(|z|) with r smooth down to 0,
// and the table holds r (times the dropout scale) for the 1664 bf16 values
// from 2^-8, below which r is constant to 5e-6 of itself, up to 32, beyond
// which act' is that of 32 in fp32.  A lookup is seven operations and one LDS
// read against 25 for the formula, and the gradient kernels are bound by
// their arithmetic.  NaN stays NaN, and an infinite z gives NaN as it does in
// the formula.
constexpr int kTabSize = 1664;
constexpr uint32_t kTabFirst = 0x3B80u;     // 2^-8

template <int ACT>
constexpr bool uses_table() { return ACT == SAG_ACT_GELU || ACT == SAG_ACT_SILU; }

template <int ACT>
__device__ __forceinline__ void build_table(float* tab, float scale, int t, int threads) {
    if constexpr (uses_table<ACT>()) {
        for (int i = t; i < kTabSize; i += threads) {
            const float a = __uint_as_float((kTabFirst + i) << 16);
            tab[i] = (act_grad<ACT>(a, 0.f) - 0.5f) * scale / a;
        }
        __syncthreads();
    }
}

// scale act'(z) for the bf16 bits in the high half of `zbits` (the low half
// is 0); half = scale / 2.
__device__ __forceinline__ float table_grad(const float* tab, uint32_t zbits, float half) {
    const float z = __uint_as_float(zbits);
    uint32_t i = (zbits >> 16) & 0x7fffu;
    i = i < kTabFirst ? kTabFirst : (i > kTabFirst + kTabSize - 1 ? kTabFirst + kTabSize - 1 : i);
    return fmaf(__builtin_amdgcn_fmed3f(z, -32.f, 32.f), tab[i - kTabFirst], fmaf(z, 0.f, half));
}

// The eight values of dZ = act'(Z) dropout(G) from the vectors of G and Z.
template <int ACT, bool DROP>
__device__ __forceinline__ void dz_of(u32x4_t g, u32x4_t z, const float* tab, const DropArgs& drop, uint32_t node,
                                      uint32_t block, uint32_t call, float slope, float (&f)[8]) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if constexpr (DROP) drop.draws(node, block, call, w);
    const float half = DROP ? 0.5f * drop.scale : 0.5f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        // (two at a time: all eight's temporaries at once cost a wavefront a SIMD)
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 2 * q; e < 2 * q + 2; ++e) {
            float x = __uint_as_float(e & 1 ? g[q] & 0xffff0000u : g[q] << 16);
            const uint32_t zb = e & 1 ? z[q] & 0xffff0000u : z[q] << 16;
            if constexpr (uses_table<ACT>()) x *= table_grad(tab, zb, half);
            else if constexpr (ACT != SAG_ACT_NONE) x = times_act_grad<ACT>(x, __uint_as_float(zb), slope);
            // (last: a dropped value is 0 whatever G and Z are; the table has the scale)
            if constexpr (DROP) x = uses_table<ACT>() ? drop.mask(x, w, e) : drop.apply(x, w, e);
            f[e] = x;
        }
    }
}

__device__ __forceinline__ u32x4_t pack8(const float (&f)[8]) {
    return u32x4_t{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
}

template <class T>
struct NnArgs {
    const T* a;           // GRAD: G
    int64_t lda, M, K;
    const T* az;          // GRAD: Z
    int64_t ldaz;
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
    float out_scale = 1.f;   // of the stored values (a backward product of unscaled dZ)
};

template <int BN, bool GRAD>
constexpr int nn_rows() { return GRAD && BN > 64 ? 64 : 128; }

// WM x WN wavefronts, each MB x NB blocks of 32 x 32.  GRAD (bf16, 256
// columns): A is dZ, computed from G and Z on its way into LDS and stored
// nowhere, once per row as long as the columns make one block; the epilogue
// only stores.
template <class T, int BN, int ACT, bool DROP, bool GRAD>
__global__ __launch_bounds__((BN == 256 ? 512 : 256), GRAD ? (BN == 256 ? 4 : 3) : 1) void dense_nn(NnArgs<T> p) {
    constexpr int kThreads = BN == 256 ? 512 : 256, kBM = nn_rows<BN, GRAD>();
    constexpr int V = Vec<T>::N;
    constexpr int CK = kRowB / static_cast<int>(sizeof(T));
    constexpr int WN = BN >= 128 ? BN / 64 : 1, WM = kThreads / 64 / WN;
    constexpr int MB = kBM / WM / 32, NB = BN / WN / 32;
    constexpr int UA = kBM * 8 / kThreads, UB = BN * 8 / kThreads;   // 16-byte units per thread
    constexpr int kTiles = (kBM + BN) * kRowB;
    constexpr int kStage = kThreads / 64 * 32 * kStagePitch;
    __shared__ __attribute__((aligned(16))) unsigned char lds[kTiles > kStage ? kTiles : kStage];
    unsigned char* As = lds;
    unsigned char* Bs = lds + kBM * kRowB;

    __shared__ float tab[GRAD && uses_table<ACT>() ? kTabSize : 1];
    if constexpr (GRAD) build_table<ACT>(tab, DROP ? p.drop.scale : 1.f, threadIdx.x, kThreads);
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const int h = lane >> 5, l32 = lane & 31;
    const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t m0 = tile / p.n_blk * kBM, n0 = tile % p.n_blk * BN;

    u32x4_t ra[UA], rz[GRAD ? UA : 1], rb[UB];
    uint32_t node[GRAD && DROP ? UA : 1], call = 0;
    if constexpr (DROP) call = p.drop.call_now();
    if constexpr (GRAD && DROP) {
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const int64_t row = m0 + (t + i * kThreads) / 8;
            node[i] = p.drop.node_of(row < p.M ? row : p.M - 1);
        }
    }
    const int64_t last = (p.K + V - 1) / V * V - V;
    auto load = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const int q = t + i * kThreads, r = q >> 3, u = q & 7;
            const int64_t row = m0 + r < p.M ? m0 + r : p.M - 1;
            const int64_t k = k0 + u * V;
            ra[i] = load16(p.a + row * p.lda + (k < last ? k : last));
            if constexpr (GRAD && ACT != SAG_ACT_NONE) rz[i] = load16(p.az + row * p.ldaz + (k < last ? k : last));
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
            if constexpr (GRAD) {
                float f[8];
                dz_of<ACT, DROP>(ra[i], rz[ACT == SAG_ACT_NONE ? 0 : i], tab, p.drop, node[DROP ? i : 0],
                                 static_cast<uint32_t>((k0 >> 3) + u), call, p.slope, f);
                ra[i] = pack8(f);
            }
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
            // (independent sums in turn: a product waits for the one before it into the same sum)
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b[j]),
                                                                             __builtin_bit_cast(bf16x8_t, a[i]),
                                                                             acc[i][j], 0, 0, 0);
            } else {
                // unit h holds k 4h .. 4h + 3 of the step: product q pairs k q with k 4 + q
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(f32x4_t, b[j])[q],
                                                                             __builtin_bit_cast(f32x4_t, a[i])[q],
                                                                             acc[i][j], 0, 0, 0);
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
            if (!GRAD && p.res) rv.load(p.res + row * p.ldr + col, live);
            const float4 lo = *reinterpret_cast<const float4*>(st + r * kStagePitch + u * 32);
            const float4 hi = *reinterpret_cast<const float4*>(st + r * kStagePitch + u * 32 + 16);
            float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += bias[e];
            if (!GRAD && p.z) Eight<T>::put(p.z + row * p.ldz + col, y, live);
            if constexpr (!GRAD) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = ACT == SAG_ACT_NONE && !DROP ? y[e] * p.out_scale : act_value<ACT, T>(y[e], p.slope);
            }
            if constexpr (DROP && !GRAD) {
                uint32_t dw[4];
                p.drop.draws(p.drop.node_of(row), static_cast<uint32_t>(col >> 3), call, dw);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = p.drop.apply(y[e], dw, e);
            }
            if (!GRAD && p.res) {
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

// ---- few tiles ---------------------------------------------------------------------------
// The same product where 32 x 32 tiles do not fill the chip: a workgroup of
// up to sixteen wavefronts does one tile (of 32 x 32, or 16 x 16), each
// wavefront every sixteenth piece of k, 128 bytes (256), and their sums are added in LDS in a fixed tree before
// the epilogue.  Operands go from memory straight into the matrix cores'
// registers, B from the weight as it lies (two bytes or four a load for the
// forward product, whole vectors along the rows for the gradient's), so there
// is one launch, no workspace and one round of loads in front of the products.
// What bounds it is latency: launch, one memory round trip and the tree.
constexpr int kSmallTiles = 128;           // up to half as many as CUs: see small_tiles
constexpr int kFewTiles = 512;             // taken up to two workgroups a CU

// Sixteen bytes from an address aligned to an element.
template <class T>
__device__ __forceinline__ u32x4_t load16_any(const T* p) {
    struct __attribute__((packed, aligned(sizeof(T)))) Any { u32x4_t v; };
    return reinterpret_cast<const Any*>(p)->v;
}

template <int TE> constexpr int few_pitch() { return TE + 4; }             // floats of a tile row in LDS
template <class T, int TE> constexpr int few_piece() { return 4 * (64 / TE) * Vec<T>::N; }   // k a wavefront takes at once

template <class T, int ACT, bool DROP, bool GRAD, int TE>
__global__ __launch_bounds__(1024) void dense_few(NnArgs<T> p, const T* __restrict__ w, int64_t ldw) {
    constexpr int V = Vec<T>::N, CK = few_piece<T, TE>(), PITCH = few_pitch<TE>();
    extern __shared__ __attribute__((aligned(16))) float part[];   // [wavefront][TE][PITCH]
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, waves = blockDim.x >> 6;
    const int h = lane / TE, lt = lane % TE;
    const uint32_t tm = blockIdx.x / static_cast<uint32_t>(p.n_blk), tn = blockIdx.x % static_cast<uint32_t>(p.n_blk);
    const int64_t m0 = static_cast<int64_t>(tm) * TE, n0 = static_cast<int64_t>(tn) * TE;
    const int64_t row = m0 + lt < p.M ? m0 + lt : p.M - 1, col = n0 + lt < p.N ? n0 + lt : p.N - 1;
    uint32_t call = 0, node = 0;
    if constexpr (DROP) call = p.drop.call_now();
    if constexpr (DROP && GRAD) node = p.drop.node_of(row);
    const T* ar = p.a + row * p.lda;
    const T* zr = GRAD && ACT != SAG_ACT_NONE ? p.az + row * p.ldaz : nullptr;
    std::conditional_t<TE == 32, f32x16_t, f32x4_t> acc;
#pragma unroll
    for (int r = 0; r < TE * TE / 64; ++r) acc[r] = 0.f;
    for (int64_t k0 = static_cast<int64_t>(wave) * CK; k0 < p.K; k0 += static_cast<int64_t>(waves) * CK) {
        u32x4_t a[4], z[4], b[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // this lane's V values of k, the last piece's padded with zeros
            const int64_t k = k0 + s * (CK / 4) + h * V;
            const int left = p.K - k >= V ? V : (p.K > k ? static_cast<int>(p.K - k) : 0);
            const int64_t ka = left ? k : 0;
            a[s] = load16(ar + ka);
            if constexpr (GRAD && ACT != SAG_ACT_NONE) z[s] = load16(zr + ka);
            if constexpr (GRAD) {
                // W's row `col` along k
                const T* wr = w + col * ldw + ka;
                if (left == V) {
                    b[s] = load16_any(wr);
                } else {
                    b[s] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        uint32_t x = 0u;
                        if (e < left) {
                            if constexpr (sizeof(T) == 2) x = static_cast<uint32_t>(wr[e]) << (16 * (e & 1));
                            else x = __float_as_uint(wr[e]);
                        }
                        b[s][e * static_cast<int>(sizeof(T)) / 4] |= x;
                    }
                }
            } else {
                // V rows of W at column `col`
                b[s] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const T x = w[(e < left ? k + e : 0) * ldw + col];
                    if constexpr (sizeof(T) == 2) b[s][e / 2] |= (e < left ? static_cast<uint32_t>(x) : 0u) << (16 * (e & 1));
                    else b[s][e] = e < left ? __float_as_uint(x) : 0u;
                }
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int64_t k = k0 + s * (CK / 4) + h * V;
            const int left = p.K - k >= V ? V : (p.K > k ? static_cast<int>(p.K - k) : 0);
            if constexpr (GRAD) {
                float f[V];
                unpack<T>(as_uint4(a[s]), f);
                if constexpr (ACT != SAG_ACT_NONE) {
                    float zf[V];
                    unpack<T>(as_uint4(z[s]), zf);
#pragma unroll
                    for (int e = 0; e < V; ++e) f[e] = times_act_grad<ACT>(f[e], zf[e], p.slope);
                }
                if constexpr (DROP) {
                    uint32_t dw[4];
                    p.drop.draws(node, static_cast<uint32_t>(k >> 3), call, dw);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        // (four fp32 columns are one half of a block's eight)
                        if constexpr (V == 8) f[e] = p.drop.apply(f[e], dw, e);
                        else f[e] = h & 1 ? p.drop.apply(f[e], dw, e + 4) : p.drop.apply(f[e], dw, e);
                    }
                }
                if constexpr (V == 8) a[s] = u32x4_t{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
                else a[s] = u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
            }
            if (left < V) a[s] = keep_first<T>(a[s], left);
            if constexpr (sizeof(T) == 2) {
                const bf16x8_t bb = __builtin_bit_cast(bf16x8_t, b[s]), aa = __builtin_bit_cast(bf16x8_t, a[s]);
                if constexpr (TE == 32) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bb, aa, acc, 0, 0, 0);
                else acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bb, aa, acc, 0, 0, 0);
            } else {
                const f32x4_t bb = __builtin_bit_cast(f32x4_t, b[s]), aa = __builtin_bit_cast(f32x4_t, a[s]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (TE == 32) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bb[q], aa[q], acc, 0, 0, 0);
                    else acc = __builtin_amdgcn_mfma_f32_16x16x4f32(bb[q], aa[q], acc, 0, 0, 0);
                }
            }
        }
    }
    float* mine = part + wave * TE * PITCH;
#pragma unroll
    for (int q = 0; q < TE * TE / 256; ++q)
        *reinterpret_cast<float4*>(mine + lt * PITCH + 8 * q + 4 * h) =
            make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
    __syncthreads();
    // units of eight columns, four lanes to a unit, each every fourth wavefront's sum
    for (int unit = t >> 2; unit < TE * TE / 8; unit += blockDim.x >> 2) {
        const int r = unit / (TE / 8), u = unit % (TE / 8);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.f;
        for (int v = t & 3; v < waves; v += 4) {
            const float* src = part + (v * TE + r) * PITCH + u * 8;
            const float4 lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + 4);
            y[0] += lo.x; y[1] += lo.y; y[2] += lo.z; y[3] += lo.w;
            y[4] += hi.x; y[5] += hi.y; y[6] += hi.z; y[7] += hi.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] += __shfl_xor(y[e], 1, 64);
            y[e] += __shfl_xor(y[e], 2, 64);
        }
        const int64_t orow = m0 + r, ocol = n0 + u * 8;
        const int live = p.N - ocol < 8 ? static_cast<int>(p.N - ocol) : 8;
        if ((t & 3) || orow >= p.M || live <= 0) continue;
        if constexpr (!GRAD) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += p.bias && e < live ? p.bias[ocol + e] : 0.f;
            if (p.z) Eight<T>::put(p.z + orow * p.ldz + ocol, y, live);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = act_value<ACT, T>(y[e], p.slope);
            if constexpr (DROP) {
                uint32_t dw[4];
                p.drop.draws(p.drop.node_of(orow), static_cast<uint32_t>(ocol >> 3), call, dw);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = p.drop.apply(y[e], dw, e);
            }
            if (p.res) {
                Eight<T> rv;
                rv.load(p.res + orow * p.ldr + ocol, live);
                float f[8];
                rv.get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += f[e];
            }
        }
        Eight<T>::put(p.out + orow * p.ldo + ocol, y, live);
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
    if constexpr (ACT != SAG_ACT_NONE) {
        float zf[8];
        zv.get(zf);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = times_act_grad<ACT>(f[e], zf[e], slope);
    }
    if (drop.T) {
        uint32_t dw[4];
        drop.draws(drop.node_of(row), static_cast<uint32_t>(u), drop.call_now(), dw);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = drop.apply(f[e], dw, e);
    }
    Eight<T>::put(hi + row * ldh + col, f, live);
    if (lo) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = f[e] - to_f32(from_f32<T>(f[e]));
        Eight<T>::put(lo + row * ldh + col, r, live);
    }
}

// ---- dW (bf16) ---------------------------------------------------------------------------
// C[K, N] = X^T dZ: a workgroup takes 256 rows of C (columns of X) by 128
// columns and a run of rows of X, 32 rows a step through LDS (two stages, one
// barrier a step; the next step's loads in registers), and leaves its
// fp32 sums as a partial; dense_tn_reduce adds the partials in order.  The
// matrix cores reduce over rows, so both operands come out of the row-major
// tiles by the LDS transpose read ds_read_b64_tr_b16 (for four rows and
// sixteen columns lane i of sixteen gets column i of the four rows).
// A bf16 dZ alone would put 2^-8 into every term of an fp32 result, so dZ is
// held as two bf16 parts (PARTS) and multiplied twice: 2^-16 a term, 2.4e-6
// of the result in the 2-norm, which is what fp32 sums of 50,000 terms are off
// by.  Below kFineRows rows a third part takes that to 1e-7.  Its tiles leave
// LDS room for one stage instead of two (the whole backward pass with GELU, two
// parts -> three: 2700 x 256 -> 256 29.1 us both, 32767 x 256 -> 256 49 -> 53,
// 10000 x 602 -> 128 38 -> 40, 10000 x 1500 -> 512, which computes dZ once a
// block of 256 inputs, 118 -> 158).  Without an activation or with ReLU, dZ is
// G or 0 exactly, up to the dropout scale, which the reduction applies.  FROM_G: dZ comes from G and Z (z); otherwise hi and lo
// are read.  Column sums (db) are taken of the fp32 dZ on its way into LDS.
constexpr int kTnWaves = 16, kTnThreads = kTnWaves * 64, kTnK = 256, kTnN = 128, kTnRows = 64;
constexpr int64_t kFineRows = 32768;
constexpr int kTnPX = kTnK * 2 + 64, kTnPZ = kTnN * 2 + 64;     // row pitches in LDS: 16 banks a row apart

struct TnArgs {
    const uint16_t* x;
    int64_t ldx, M, K, N;
    const uint16_t* g;          // FROM_G: G, else hi
    int64_t ldg;
    const uint16_t* z;          // FROM_G: Z, else lo
    int64_t ldz;
    float slope;
    DropArgs drop;
    int64_t n_kblk, n_nblk, rows_per_chunk;
    float* part;                // [chunk][n_kblk * 256][n_nblk * 128]
    float* part_cs;             // [chunk][n_nblk * 128], nullable
};

template <int ACT>
constexpr bool dz_exact() { return ACT == SAG_ACT_NONE || ACT == SAG_ACT_RELU; }

template <int ACT, bool DROP, int PARTS, bool FROM_G>
__global__ __launch_bounds__(kTnThreads, 4) void dense_tn(TnArgs p) {
    typedef short i16x4_t __attribute__((ext_vector_type(4)));
    constexpr int SX = kTnRows * kTnPX, SZ = kTnRows * kTnPZ;
    constexpr int STAGE = SX + PARTS * SZ, STAGES = PARTS == 3 ? 1 : 2;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    float* tab = reinterpret_cast<float*>(lds + STAGES * STAGE);
    if constexpr (FROM_G) build_table<ACT>(tab, DROP ? p.drop.scale : 1.f, threadIdx.x, kTnThreads);
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wk = wave >> 2, wn = wave & 3;
    // the blocks of one chunk next to each other on one XCD
    const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t nb = tile % p.n_nblk, kb = tile / p.n_nblk % p.n_kblk, chunk = tile / (p.n_nblk * p.n_kblk);
    const int64_t k0 = kb * kTnK, n0 = nb * kTnN;
    const int64_t m_begin = chunk * p.rows_per_chunk;
    const int64_t m_end = m_begin + p.rows_per_chunk < p.M ? m_begin + p.rows_per_chunk : p.M;

    // this thread's units: two of X (rows t / 32 and 32 more), one of dZ
    const int xr = t >> 5, xc = (t & 31) * 8, zr = t >> 4, zc = (t & 15) * 8;
    const int64_t xlast = (p.K + 7) / 8 * 8 - 8, zlast = (p.N + 7) / 8 * 8 - 8;
    const int64_t xcol = k0 + xc < xlast ? k0 + xc : xlast, zcol = n0 + zc < zlast ? n0 + zc : zlast;
    const uint32_t block = static_cast<uint32_t>((n0 + zc) >> 3);
    uint32_t call = 0;
    if constexpr (DROP && FROM_G) call = p.drop.call_now();
    u32x4_t rx[2], rg, rz;
    uint32_t node = 0;
    // the rows of the step that is loaded next; a row past the chunk is read
    // from the operand's first, and not used
    const char* px = reinterpret_cast<const char*>(p.x + (m_begin + xr) * p.ldx + xcol);
    const char* pg = reinterpret_cast<const char*>(p.g + (m_begin + zr) * p.ldg + zcol);
    const char* pz = reinterpret_cast<const char*>(p.z + (m_begin + zr) * p.ldz + zcol);
    const int64_t half_x = 64 * p.ldx, step_g = 128 * p.ldg, step_z = 128 * p.ldz;   // bytes: 32 rows, 64 rows
    constexpr bool kReadZ = FROM_G ? ACT != SAG_ACT_NONE : PARTS == 2;
    auto load = [&](int64_t m) __attribute__((always_inline)) {
        rx[0] = load16(m + xr < m_end ? px : reinterpret_cast<const char*>(p.x));
        rx[1] = load16(m + xr + 32 < m_end ? px + half_x : reinterpret_cast<const char*>(p.x));
        px += 2 * half_x;
        const bool in = m + zr < m_end;
        rg = load16(in ? pg : reinterpret_cast<const char*>(p.g));
        pg += step_g;
        if constexpr (kReadZ) {
            rz = load16(in ? pz : reinterpret_cast<const char*>(p.z));
            pz += step_z;
        }
        if constexpr (DROP && FROM_G) node = p.drop.node_of(in ? m + zr : m_begin);
    };
    float cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 0.f;
    // (rows past the chunk are written as zeros, in both operands: a clamped
    // row of X may hold infinities)
    auto store = [&](int st, int64_t m) __attribute__((always_inline)) {
        unsigned char* Xs = lds + st * STAGE;
        unsigned char* Hs = Xs + SX;
        const u32x4_t none = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            store16(Xs + (xr + 32 * i) * kTnPX + xc * 2, m + xr + 32 * i < m_end ? rx[i] : none);
        const bool in = m + zr < m_end;
        if constexpr (FROM_G) {
            float f[8];
            dz_of<ACT, DROP>(rg, rz, tab, p.drop, node, block, call, p.slope, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = in ? f[e] : 0.f;
                cs[e] += f[e];
            }
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                const u32x4_t part = pack8(f);
                store16(Hs + q * SZ + zr * kTnPZ + zc * 2, part);
                if (q + 1 < PARTS) {
                    float hf[8];
                    unpack<uint16_t>(as_uint4(part), hf);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] -= hf[e];
                }
            }
        } else {
            const u32x4_t hi = in ? rg : none, lo = PARTS == 2 && in ? rz : none;
            float f[8];
            unpack<uint16_t>(as_uint4(hi), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] += f[e];
            store16(Hs + zr * kTnPZ + zc * 2, hi);
            if constexpr (PARTS == 2) {
                unpack<uint16_t>(as_uint4(lo), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) cs[e] += f[e];
                store16(Hs + SZ + zr * kTnPZ + zc * 2, lo);
            }
        }
    };
    f32x16_t acc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    const int g4 = lane >> 4, q4 = (lane & 15) >> 2, r4 = lane & 3;
    auto frag = [&](const unsigned char* base, int pitch) __attribute__((always_inline)) {
        const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(base));
        const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(base + 4 * pitch));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto multiply = [&](int st) __attribute__((always_inline)) {
        const unsigned char* Xs = lds + st * STAGE;
        const unsigned char* Hs = Xs + SX;
#pragma unroll
        for (int s = 0; s < kTnRows / 16; ++s) {           // 16 rows per product
            const int m = 16 * s + 8 * (g4 >> 1) + q4, c = 16 * (g4 & 1) + 4 * r4;
            bf16x8_t xa[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) xa[i] = frag(Xs + m * kTnPX + (wk * 64 + 32 * i + c) * 2, kTnPX);
            const unsigned char* h = Hs + m * kTnPZ + (wn * 32 + c) * 2;
            // (the smallest part first)
#pragma unroll
            for (int q = PARTS - 1; q >= 0; --q) {
                const bf16x8_t y = frag(h + q * SZ, kTnPZ);
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[i], y, acc[i], 0, 0, 0);
            }
        }
    };
    const int64_t steps = (m_end - m_begin + kTnRows - 1) / kTnRows;
    load(m_begin);
    if constexpr (STAGES == 1) {
        for (int64_t s = 0; s < steps; ++s) {
            store(0, m_begin + s * kTnRows);
            load(m_begin + (s + 1) * kTnRows);
            __syncthreads();
            multiply(0);
            __syncthreads();
        }
    } else {
        store(0, m_begin);
        load(m_begin + kTnRows);
        __syncthreads();
        // step s: stage s + 1, load s + 2, multiply s (past the chunk zeros are staged)
        for (int64_t s = 0; s < steps; ++s) {
            const int cur = static_cast<int>(s & 1);
            store(cur ^ 1, m_begin + (s + 1) * kTnRows);
            load(m_begin + (s + 2) * kTnRows);
            multiply(cur);
            __syncthreads();
        }
    }
    const int64_t pn = p.n_nblk * kTnN;
    float* out = p.part + (chunk * p.n_kblk * kTnK + k0 + wk * 64 + 4 * (lane / 32)) * pn + n0 + wn * 32 + lane % 32;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            *out = acc[i][r];
            out += r % 4 == 3 ? 5 * pn : pn;
        }
    if (p.part_cs && kb == 0) {
        // the row threads of each column, in order
        float* red = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int e = 0; e < 8; ++e) red[zr * kTnN + zc + e] = cs[e];
        __syncthreads();
        if (t < kTnN) {
            float sum = 0.f;
            for (int r = 0; r < kTnRows; ++r) sum += red[r * kTnN + t];
            p.part_cs[chunk * pn + n0 + t] = sum;
        }
    }
}

// ---- dW (fp32) ---------------------------------------------------------------------------
// The same product of fp32 X and stored fp32 dZ: 128 rows of C (columns of X)
// by 32 NB WN columns, four wavefronts of WN x NB tiles of 32 x 32 each, 32
// rows a step through LDS (two stages, one barrier a step, the next step's
// loads in registers), two workgroups a CU.  The fp32 matrix instruction
// takes one value a lane and operand, adjacent lanes adjacent columns, so the
// row-major tiles are read as they lie; rows are 32 banks apart, as a lane's
// upper half reads the next row.  What bounds it is the matrix cores.
// Blocks of 128 inputs, not 256: 602 take five of them (640) where three of 256
// would be 768.  232965 x 602 -> 128: 409 us (93 TFLOP/s of products, 70% of the
// matrix cores' cycles; bytes alone would take 130).  With tiles of 32 and 64
// columns for narrow layers the whole backward pass takes, against the plain
// product's weight-gradient kernel (256 inputs a block, four times the chunks):
// 232965 x 602 -> 128 908 -> 842 us, 232965 x 562 -> 17 484 -> 387,
// 2800 x 562 -> 17 42 -> 25, 25000 x 100 -> 47 58 -> 39, 232965 x 256 -> 256 702
// -> 724.
constexpr int kT32K = 128, kT32Rows = 32, kT32PX = kT32K + 32;

struct Tn32Args {
    const float *x, *z;         // z: dZ
    int64_t ldx, ldz, M, K, N, n_kblk, n_nblk, rows_per_chunk;
    float* part;                // [chunk][n_kblk * 128][n_nblk * TN]
    float* part_cs;             // [chunk][n_nblk * TN], nullable
};

template <int NB, int WN>
__global__ __launch_bounds__(256, 2) void dense_tn32(Tn32Args p) {
    constexpr int TN = 32 * NB * WN, KB = WN, PZ = TN + 32;
    constexpr int SX = kT32Rows * kT32PX, STAGE = SX + kT32Rows * PZ;
    constexpr int UZ = TN / 32, ZT = TN / 4;        // vectors of dZ a thread, threads across its row
    __shared__ __attribute__((aligned(16))) float lds[2 * STAGE];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, h = lane >> 5, l32 = lane & 31;
    const int wk = wave / WN, wn = wave % WN;
    const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t nb = tile % p.n_nblk, kb = tile / p.n_nblk % p.n_kblk, chunk = tile / (p.n_nblk * p.n_kblk);
    const int64_t k0 = kb * kT32K, n0 = nb * TN;
    const int64_t m_begin = chunk * p.rows_per_chunk;
    const int64_t m_end = m_begin + p.rows_per_chunk < p.M ? m_begin + p.rows_per_chunk : p.M;
    const int xr = t >> 5, xc = (t & 31) * 4, zr = t / ZT, zc = t % ZT * 4;
    const int64_t xlast = (p.K + 3) / 4 * 4 - 4, zlast = (p.N + 3) / 4 * 4 - 4;
    const float* px = p.x + (k0 + xc < xlast ? k0 + xc : xlast);
    const float* pz = p.z + (n0 + zc < zlast ? n0 + zc : zlast);
    u32x4_t rx[4], rz[UZ];
    // (a row past the chunk is the chunk's first, and staged as zeros)
    auto load = [&](int64_t m) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rx[i] = load16(px + (m + xr + 8 * i < m_end ? m + xr + 8 * i : m_begin) * p.ldx);
#pragma unroll
        for (int i = 0; i < UZ; ++i) {
            const int64_t r = m + zr + 256 / ZT * i;
            rz[i] = load16(pz + (r < m_end ? r : m_begin) * p.ldz);
        }
    };
    float cs[4] = {0.f, 0.f, 0.f, 0.f};
    auto store = [&](int st, int64_t m) __attribute__((always_inline)) {
        float* Xs = lds + st * STAGE;
        float* Zs = Xs + SX;
        const u32x4_t none = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) store16(Xs + (xr + 8 * i) * kT32PX + xc, m + xr + 8 * i < m_end ? rx[i] : none);
#pragma unroll
        for (int i = 0; i < UZ; ++i) {
            const int r = zr + 256 / ZT * i;
            const u32x4_t v = m + r < m_end ? rz[i] : none;
            store16(Zs + r * PZ + zc, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) cs[e] += __uint_as_float(v[e]);
        }
    };
    f32x16_t acc[KB][NB];
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const int64_t steps = (m_end - m_begin + kT32Rows - 1) / kT32Rows;
    load(m_begin);
    store(0, m_begin);
    load(m_begin + kT32Rows);
    __syncthreads();
    // step s: stage s + 1, load s + 2, multiply s (past the chunk zeros are staged)
    for (int64_t s = 0; s < steps; ++s) {
        const int cur = static_cast<int>(s & 1);
        store(cur ^ 1, m_begin + (s + 1) * kT32Rows);
        load(m_begin + (s + 2) * kT32Rows);
        const float* Xs = lds + cur * STAGE + h * kT32PX + wk * 32 * KB + l32;
        const float* Zs = lds + cur * STAGE + SX + h * PZ + wn * 32 * NB + l32;
#pragma unroll
        for (int q = 0; q < kT32Rows / 2; ++q) {
            float a[KB], b[NB];
#pragma unroll
            for (int i = 0; i < KB; ++i) a[i] = Xs[2 * q * kT32PX + 32 * i];
#pragma unroll
            for (int j = 0; j < NB; ++j) b[j] = Zs[2 * q * PZ + 32 * j];
#pragma unroll
            for (int i = 0; i < KB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[j], acc[i][j], 0, 0, 0);
        }
        __syncthreads();
    }
    const int64_t pn = p.n_nblk * TN;
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            float* out = p.part + (chunk * p.n_kblk * kT32K + k0 + (wk * KB + i) * 32 + 4 * h) * pn + n0 + (wn * NB + j) * 32 + l32;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                *out = acc[i][j][r];
                out += r % 4 == 3 ? 5 * pn : pn;
            }
        }
    if (p.part_cs && kb == 0) {
        // the row threads of each column, in order
#pragma unroll
        for (int e = 0; e < 4; ++e) lds[zr * TN + zc + e] = cs[e];
        __syncthreads();
        if (t < TN) {
            float sum = 0.f;
            for (int r = 0; r < 256 / ZT; ++r) sum += lds[r * TN + t];
            p.part_cs[chunk * pn + n0 + t] = sum;
        }
    }
}

// dW and db: the partials in chunk order, four threads to an element, each a
// quarter of the chunks, eight loads ahead; times the dropout scale where the
// sums are of G itself.
__global__ __launch_bounds__(256) void dense_tn_reduce(const float* __restrict__ part, const float* __restrict__ part_cs,
                                                       int64_t chunks, int64_t K, int64_t N, int64_t pk, int64_t pn,
                                                       float scale, float* __restrict__ dW, float* __restrict__ db) {
    __shared__ float sh[256];
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
    const int quarter = threadIdx.x >> 6;
    const int64_t total = (dW ? K * N : 0) + (db ? N : 0);
    const float* src = part;
    int64_t stride = pk * pn;
    float* dst = nullptr;
    if (idx < total) {
        if (dW && idx < K * N) {
            src = part + idx / N * pn + idx % N;
            dst = dW + idx;
        } else {
            const int64_t n = idx - (dW ? K * N : 0);
            src = part_cs + n;
            stride = pn;
            dst = db + n;
        }
    }
    const int64_t per = (chunks + 3) / 4, lo = quarter * per, hi = lo + per < chunks ? lo + per : chunks;
    float s = 0.f;
    if (dst) {
        int64_t c = lo;
        for (; c + 8 <= hi; c += 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = src[(c + u) * stride];
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
        for (; c < hi; ++c) s += src[c * stride];
    }
    sh[threadIdx.x] = s;
    __syncthreads();
    if (quarter == 0 && dst) *dst = (((sh[threadIdx.x] + sh[threadIdx.x + 64]) + sh[threadIdx.x + 128]) + sh[threadIdx.x + 192]) * scale;
}

int64_t k_pad(int64_t K, sag_dtype dt) { return round_up(K, kRowB / elt_size(dt)); }
size_t pack_bytes(int64_t K, int64_t N, sag_dtype dt) {
    return static_cast<size_t>(round_up(N, 256) * k_pad(K, dt) * elt_size(dt));
}

bool few_tiles(int64_t M, int64_t N) { return cdiv(M, 32) * cdiv(N, 32) <= kFewTiles; }

// Tiles of 16 x 16 where those of 32 leave half the CUs idle or half of every
// tile empty.  They read the operands twice as often, and four times as many
// compute units read them: 2708 x 1433 -> 16 fp32 (85 tiles of 32) 15.5 -> 7.8
// us, 1000 x 512 -> 128 bf16 (128) 5.6 -> 5.2, 16000 x 256 -> 16 bf16 (500) 6.4
// -> 5.1, but 512 x 2000 -> 512 bf16 (256) 11.8 -> 21 and 4000 x 256 -> 128 fp32
// (500) 8.3 -> 11.
bool small_tiles(int64_t M, int64_t N) { return M <= 16 || N <= 16 || cdiv(M, 32) * cdiv(N, 32) <= kSmallTiles; }

// The product of few tiles; W as it lies (rows of ldw).
template <class T, bool GRAD>
sag_status few_run(const char* what, sag_act act, NnArgs<T> p, const T* w, int64_t ldw, sag_dtype dt, hipStream_t s) {
    TraceScope trace(trace_enabled() ? shape_name(what, dt == SAG_BF16 ? "bf16" : "f32", p.M, p.K, p.N) : std::string(),
                     s, elt_size(dt) * (p.M * p.K * (p.az ? 2 : 1) + p.M * p.N * (1 + (p.z ? 1 : 0) + (p.res ? 1 : 0)) + p.K * p.N),
                     2 * p.M * p.K * p.N);
    sag_status st = SAG_OK;
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto drop_c, auto edge_c) -> sag_status {
            constexpr bool DROP = decltype(drop_c)::value;
            constexpr int TE = decltype(edge_c)::value, kWaveLds = TE * few_pitch<TE>() * 4;
            static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&dense_few<T, ACT, DROP, GRAD, TE>),
                                                               hipFuncAttributeMaxDynamicSharedMemorySize, 16 * kWaveLds);
            SAG_CHECK_HIP(attr);
            p.n_blk = cdiv(p.N, TE);
            p.m_blk = cdiv(p.M, TE);
            const int64_t pieces = cdiv(p.K, few_piece<T, TE>());
            const int waves = static_cast<int>(pieces < 16 ? pieces : 16);
            dense_few<T, ACT, DROP, GRAD, TE><<<static_cast<unsigned>(p.n_blk * p.m_blk), waves * 64, waves * kWaveLds, s>>>(p, w, ldw);
            return SAG_OK;
        };
        auto edge = [&](auto drop_c) {
            return small_tiles(p.M, p.N) ? go(drop_c, std::integral_constant<int, 16>{}) : go(drop_c, std::integral_constant<int, 32>{});
        };
        st = p.drop.T ? edge(std::true_type{}) : edge(std::false_type{});
    });
    SAG_TRY(st);
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

// Packs B ([K, N]; element (k, n) at b[k sk + n sn]) and multiplies.
template <class T, bool GRAD = false>
sag_status nn_run(const char* what, sag_act act, NnArgs<T> p, const T* b, int64_t sk, int64_t sn, T* bp, sag_dtype dt,
                  hipStream_t s) {
    const int BN = GRAD && p.N > 128 ? 256 : (p.N <= 64 ? 64 : 128);
    p.Kt = k_pad(p.K, dt);
    p.bp = bp;
    p.n_blk = cdiv(p.N, BN);
    p.m_blk = cdiv(p.M, GRAD && BN > 64 ? 64 : 128);
    if (p.n_blk * p.m_blk >= (1 << 23)) return fail(SAG_E_UNSUPPORTED, std::string(what) + ": too many tiles for one launch");
    const int64_t total = p.n_blk * BN * p.Kt;
    dense_pack<T><<<dim3(static_cast<unsigned>(cdiv(total, 256))), 256, 0, s>>>(b, sk, sn, p.K, p.N, p.Kt, total, bp);
    SAG_LAUNCH_CHECK();
    const int64_t rows = p.M * p.K * (p.az ? 2 : 1) + p.M * p.N * (1 + (p.z ? 1 : 0) + (p.res ? 1 : 0));
    TraceScope trace(trace_enabled() ? shape_name(what, dt == SAG_BF16 ? "bf16" : "f32", p.M, p.K, p.N) : std::string(),
                     s, elt_size(dt) * (rows + p.K * p.N), 2 * p.M * p.K * p.N);
    const dim3 grid(static_cast<unsigned>(p.n_blk * p.m_blk));
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
        auto go = [&](auto bn) {
            constexpr int BN = decltype(bn)::value;
            constexpr int NT = BN == 256 ? 512 : 256;
            if (p.drop.T) dense_nn<T, BN, ACT, true, GRAD><<<grid, NT, 0, s>>>(p);
            else dense_nn<T, BN, ACT, false, GRAD><<<grid, NT, 0, s>>>(p);
        };
        if (BN == 64) go(std::integral_constant<int, 64>{});
        else if (BN == 128) go(std::integral_constant<int, 128>{});
        if constexpr (GRAD) {
            if (BN == 256) go(std::integral_constant<int, 256>{});
        }
    });
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

template <class T>
sag_status forward_typed(NnArgs<T> p, const void* W, sag_act act, sag_dtype dt, void* ws, hipStream_t s) {
    const T* w = static_cast<const T*>(W);
    if (few_tiles(p.M, p.N)) return few_run<T, false>("dense", act, p, w, p.N, dt, s);
    return nn_run<T>("dense", act, p, w, p.N, 1, static_cast<T*>(ws), dt, s);
}

// ---- backward ------------------------------------------------------------------------------
// bf16 layers of up to 256 inputs never store dZ: the input gradient and the
// weight gradient each compute it from G and Z on its way into LDS (once a
// row, as 256 columns make one block in both).  Wider ones would compute it
// once a block of 256, where it costs more than the products (some 35 operations
// an element against 0.25 matrix operations' time a column block), so there it
// is stored first, as hi (and lo, where it is not exact); fp32, bound by the
// matrix cores, stores it as well.
bool dz_from_g(int64_t K, sag_dtype dt) { return dt == SAG_BF16 && K <= 256; }

struct TnPlan {
    int64_t tile_k, tile_n, n_kblk, n_nblk, chunks, rows_per_chunk, max_chunks;   // max_chunks: of up to M rows
};

// Columns of a tile.
int tn_cols(int64_t N, sag_dtype dt) { return dt == SAG_BF16 || N > 64 ? kTnN : (N > 32 ? 64 : 32); }

// bf16: one workgroup of sixteen wavefronts a CU; fp32: two of four.  Chunks of
// at least 128 rows.
TnPlan tn_plan(int64_t M, int64_t K, int64_t N, sag_dtype dt) {
    TnPlan p;
    p.tile_k = dt == SAG_BF16 ? kTnK : kT32K;
    p.tile_n = tn_cols(N, dt);
    p.n_kblk = cdiv(K, p.tile_k);
    p.n_nblk = cdiv(N, p.tile_n);
    const int64_t tiles = p.n_kblk * p.n_nblk, rows = dt == SAG_BF16 ? kTnRows : kT32Rows;
    int64_t want = dt == SAG_BF16 ? cdiv(256, tiles) : (tiles < 512 ? 512 / tiles : 1);
    const int64_t most = cdiv(M > 0 ? M : 1, 128);
    if (want > most) want = most;
    p.max_chunks = want;
    p.rows_per_chunk = round_up(cdiv(M > 0 ? M : 1, want), rows);
    p.chunks = cdiv(M, p.rows_per_chunk);
    return p;
}

struct BwdWs {
    void *bp, *hi, *lo;
    float *part, *part_cs;
    size_t used;
    bool fits;
};

BwdWs bwd_ws(int64_t M, int64_t K, int64_t N, sag_dtype dt, void* ws, size_t bytes) {
    Carver c(ws, bytes);
    BwdWs w{};
    w.bp = c.take<char>(pack_bytes(N, K, dt));
    if (!dz_from_g(K, dt)) w.hi = c.take<char>(dense_bytes(M, N, dt));
    if (dt == SAG_BF16 && !dz_from_g(K, dt) && M >= kFineRows) w.lo = c.take<char>(dense_bytes(M, N, dt));
    const TnPlan p = tn_plan(M, K, N, dt);
    w.part = c.take<float>(p.max_chunks * p.n_kblk * p.tile_k * p.n_nblk * p.tile_n);
    w.part_cs = c.take<float>(p.max_chunks * p.n_nblk * p.tile_n);
    w.used = c.used();
    w.fits = c.fits();
    return w;
}

template <int ACT, bool DROP, int PARTS, bool FROM_G>
sag_status launch_tn(const TnArgs& a, int64_t chunks, hipStream_t s) {
    constexpr int lds = (PARTS == 3 ? 1 : 2) * (kTnRows * kTnPX + PARTS * kTnRows * kTnPZ) +
                        (FROM_G && uses_table<ACT>() ? kTabSize * 4 : 0);
    static_assert(lds >= kTnRows * kTnN * 4, "column-sum buffer");
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&dense_tn<ACT, DROP, PARTS, FROM_G>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    SAG_CHECK_HIP(attr);
    const unsigned grid = static_cast<unsigned>(chunks * a.n_kblk * a.n_nblk);
    dense_tn<ACT, DROP, PARTS, FROM_G><<<grid, kTnThreads, lds, s>>>(a);
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

sag_status tn_join(const TnPlan& p, int64_t K, int64_t N, float scale, float* dW, float* db, const BwdWs& w, hipStream_t s) {
    const int64_t total = (dW ? K * N : 0) + (db ? N : 0);
    dense_tn_reduce<<<dim3(static_cast<unsigned>(cdiv(total, 64))), 256, 0, s>>>(
        w.part, w.part_cs, p.chunks, K, N, p.n_kblk * p.tile_k, p.n_nblk * p.tile_n, scale, dW, db);
    SAG_LAUNCH_CHECK();
    return SAG_OK;
}

// bf16: dW and db from G and Z, or from stored hi and lo.
sag_status tn_run(sag_act act, TnArgs a, bool from_g, float* dW, float* db, const BwdWs& w, hipStream_t s) {
    const TnPlan p = tn_plan(a.M, a.K, a.N, SAG_BF16);
    a.n_kblk = p.n_kblk; a.n_nblk = p.n_nblk; a.rows_per_chunk = p.rows_per_chunk;
    a.part = w.part; a.part_cs = db ? w.part_cs : nullptr;
    const bool exact = act == SAG_ACT_NONE || act == SAG_ACT_RELU;
    // a sum over G itself is scaled once, at the end
    const float scale = exact && a.drop.T ? a.drop.scale : 1.f;
    if (exact) a.drop.scale = 1.f;
    TraceScope trace(trace_enabled() ? shape_name("dense_dw", "bf16", a.M, a.K, a.N) : std::string(), s,
                     2 * (a.M * a.K + a.M * a.N * (act == SAG_ACT_NONE || (exact && !from_g) ? 1 : 2)) + 4 * (a.K * a.N + a.N),
                     (exact ? 2 : (from_g && a.M < kFineRows ? 6 : 4)) * a.M * a.K * a.N);
    if (p.chunks) {
        sag_status st = SAG_OK;
        if (!from_g) {
            st = exact ? launch_tn<SAG_ACT_NONE, false, 1, false>(a, p.chunks, s)
                       : launch_tn<SAG_ACT_NONE, false, 2, false>(a, p.chunks, s);
        } else {
            with_act(act, [&](auto ac) {
                constexpr int ACT = decltype(ac)::value;
                auto go = [&](auto parts) {
                    constexpr int PARTS = decltype(parts)::value;
                    return a.drop.T ? launch_tn<ACT, true, PARTS, true>(a, p.chunks, s)
                                    : launch_tn<ACT, false, PARTS, true>(a, p.chunks, s);
                };
                if constexpr (dz_exact<ACT>()) st = go(std::integral_constant<int, 1>{});
                else if (a.M < kFineRows) st = go(std::integral_constant<int, 3>{});
                else st = go(std::integral_constant<int, 2>{});
            });
        }
        SAG_TRY(st);
    }
    return tn_join(p, a.K, a.N, scale, dW, db, w, s);
}

// fp32: dW and db from X and the stored dZ.
sag_status tn32_run(Tn32Args a, float* dW, float* db, const BwdWs& w, hipStream_t s) {
    const TnPlan p = tn_plan(a.M, a.K, a.N, SAG_F32);
    a.n_kblk = p.n_kblk; a.n_nblk = p.n_nblk; a.rows_per_chunk = p.rows_per_chunk;
    a.part = w.part; a.part_cs = db ? w.part_cs : nullptr;
    TraceScope trace(trace_enabled() ? shape_name("dense_dw", "f32", a.M, a.K, a.N) : std::string(), s,
                     4 * (a.M * a.K + a.M * a.N + a.K * a.N + a.N), 2 * a.M * a.K * a.N);
    if (p.chunks) {
        const unsigned grid = static_cast<unsigned>(p.chunks * p.n_kblk * p.n_nblk);
        if (p.tile_n == 128) dense_tn32<2, 2><<<grid, 256, 0, s>>>(a);
        else if (p.tile_n == 64) dense_tn32<1, 2><<<grid, 256, 0, s>>>(a);
        else dense_tn32<1, 1><<<grid, 256, 0, s>>>(a);
        SAG_LAUNCH_CHECK();
    }
    return tn_join(p, a.K, a.N, 1.f, dW, db, w, s);
}

template <class T>
sag_status backward_typed(int64_t M, const T* X, int64_t ldx, int64_t K, const T* W, int64_t N, sag_act act, float slope,
                          const DropArgs& drop, const T* Z, int64_t ldz, const T* G, int64_t ldg, float* dW, float* db,
                          T* dX, int64_t ldd, sag_dtype dt, const BwdWs& w, hipStream_t s) {
    const int64_t ldh = ldv(N, dt), upr = cdiv(N, 8);
    const bool from_g = dz_from_g(K, dt), exact = act == SAG_ACT_NONE || act == SAG_ACT_RELU;
    T* hi = static_cast<T*>(w.hi);
    T* lo = exact ? nullptr : static_cast<T*>(w.lo);
    // the weight gradient of few rows takes three parts of dZ, which are made of G and Z
    const bool dw_from_g = from_g || (dt == SAG_BF16 && !exact && M < kFineRows);
    // (the tiled input gradient reads a stored dZ, and so does the weight gradient)
    if (M > 0 && !from_g && ((dX && !few_tiles(M, K)) || (!dw_from_g && (dW || db)))) {
        const int64_t blocks = cdiv(M * upr, kThreads);
        if (blocks >= (1 << 24)) return fail(SAG_E_UNSUPPORTED, "dense backward: too many elements for one launch");
        TraceScope trace(trace_enabled() ? shape_name("dense_dz", dt == SAG_BF16 ? "bf16" : "f32", M, N, 0) : std::string(),
                         s, elt_size(dt) * M * N * (2 + (act != SAG_ACT_NONE ? 1 : 0) + (lo ? 1 : 0)), 0);
        // (exact in bf16: G or 0, the products take the dropout scale)
        DropArgs unscaled = drop;
        if (exact && dt == SAG_BF16) unscaled.scale = 1.f;
        with_act(act, [&](auto ac) {
            dense_dz<T, decltype(ac)::value><<<dim3(static_cast<unsigned>(blocks)), kThreads, 0, s>>>(
                M, N, upr, Z, ldz, G, ldg, slope, unscaled, hi, lo, ldh);
        });
        SAG_LAUNCH_CHECK();
    }
    if (dX && M > 0) {
        NnArgs<T> p{};
        p.M = M; p.K = N; p.N = K;
        p.out = dX; p.ldo = ldd;
        if (few_tiles(M, K)) {
            p.a = G; p.lda = ldg; p.az = act == SAG_ACT_NONE ? nullptr : Z; p.ldaz = ldz;
            p.slope = slope; p.drop = drop;
            SAG_TRY((few_run<T, true>("dense_dx", act, p, W, N, dt, s)));
        } else if (from_g) {
            if constexpr (sizeof(T) == 2) {
                p.a = G; p.lda = ldg; p.az = act == SAG_ACT_NONE ? nullptr : Z; p.ldaz = ldz;
                p.slope = slope; p.drop = drop;
                SAG_TRY((nn_run<T, true>("dense_dx", act, p, W, 1, N, static_cast<T*>(w.bp), dt, s)));
            }
        } else {
            p.a = hi; p.lda = ldh;
            p.out_scale = exact && dt == SAG_BF16 && drop.T ? drop.scale : 1.f;
            SAG_TRY(nn_run<T>("dense_dx", SAG_ACT_NONE, p, W, 1, N, static_cast<T*>(w.bp), dt, s));
        }
    }
    if (!dW && !db) return SAG_OK;
    if constexpr (sizeof(T) == 2) {
        TnArgs a{};
        a.x = X; a.ldx = ldx; a.M = M; a.K = K; a.N = N; a.slope = slope; a.drop = drop;
        a.g = dw_from_g ? G : hi; a.ldg = dw_from_g ? ldg : ldh;
        a.z = dw_from_g ? Z : lo; a.ldz = dw_from_g ? ldz : ldh;
        return tn_run(act, a, dw_from_g, dW, db, w, s);
    } else {
        Tn32Args a{};
        a.x = X; a.ldx = ldx; a.z = hi; a.ldz = ldh; a.M = M; a.K = K; a.N = N;
        return tn32_run(a, dW, db, w, s);
    }
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
    if (M < 0 || K < 1 || N < 1 || (dt != SAG_F32 && dt != SAG_BF16) || few_tiles(M, N)) return 0;
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
    const size_t need = sag_dense_forward_workspace_bytes(M, K, N, dt);
    if (need && (!ws || !aligned16(ws) || ws_bytes < need))
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
