// Matrix products over lists: the caller's (alpha op(a) op(b) + beta c), and those
// of the Newton-Schulz steps.
#include "adamw_math.h"
#include "matrices.h"
#include "mfma_tile.h"

namespace zs {
namespace {

constexpr int kRowsAtOnce = 4;
using T256 = Tile<256, 256, 2, 4, 2>;
using T128 = Tile<128, 128, 2, 2, 2>;
using T64 = Tile<64, 64, 2, 2, 3>;

// The tile that workgroup w of a launch runs.  gfx950 deals workgroups to its 8
// XCDs in turn: runs of as many consecutive tiles as an XCD works on at a time
// go to one XCD, whose L2 then holds the rows and columns that they share.
template <class T>
__device__ __forceinline__ uint32_t tile_of(uint32_t w, uint32_t n) {
    constexpr uint32_t kRun = T::BM == 256 ? 32 : T::BM == 128 ? 64 : 128, kAll = 8 * kRun;
    const uint32_t base = w / kAll * kAll, i = w - base;
    if (base + kAll <= n) return base + (i % 8) * kRun + i / 8;
    return base + (uint32_t)xcd_slot(i, n - base);
}

// Tile t of a matrix of tm x tn tiles, as its row and column: panels of 8 columns,
// in them bands of 4 rows.  An XCD's 32 tiles share 4 rows and 8 columns of operands,
// and the 8 XCDs' together 16 and 16 of a matrix of 16 rows: the wider operand
// comes from memory once (against bands over all columns, 4096 x 88064 x 4096:
// 1170 -> 1218 TFLOP/s).
__device__ __forceinline__ void tile_in_bands(uint32_t t, uint32_t tm, uint32_t tn, uint32_t& i, uint32_t& j) {
    constexpr uint32_t kPanel = 8, kBand = 4;
    const uint32_t panel = t / (kPanel * tm), columns = min(kPanel, tn - panel * kPanel), in = t - panel * kPanel * tm;
    const uint32_t band = in / (kBand * columns), rows = min(kBand, tm - band * kBand), at = in - band * kBand * columns;
    i = band * kBand + at % rows;
    j = panel * kPanel + at / rows;
}
// Tile t of a triangle: row i has i + 1 of them.
__device__ __forceinline__ void tile_in_triangle(uint32_t t, uint32_t& i, uint32_t& j) {
    uint32_t r = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > t) --r;
    while ((r + 1) * (r + 2) / 2 <= t) ++r;
    i = r;
    j = t - r * (r + 1) / 2;
}

// Calls f(row, column, x) for every eight neighbouring columns' values x[8] that this
// lane has of a tile.
template <class T, bool BCOLS, class F>
__device__ __forceinline__ void each_row(const f32x4 (&acc)[T::MI][T::NI], int m0, int n0, F&& f) {
    int row, column;
    lane_place<T>(m0, n0, row, column);
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int u = 0; u < T::NI / 2; ++u) {
            f32x4 p[2];
            pair_of<T, BCOLS>(acc, i, u, p);
            float x[8] = {p[0].x, p[0].y, p[0].z, p[0].w, p[1].x, p[1].y, p[1].z, p[1].w};
            f(row + i, column + 32 * u, x);
        }
}
// Calls f(row, column, x) for every MI neighbouring rows' values x[MI] of one column.
template <class T, bool BCOLS, class F>
__device__ __forceinline__ void each_column(const f32x4 (&acc)[T::MI][T::NI], int m0, int n0, F&& f) {
    int row, column;
    lane_place<T>(m0, n0, row, column);
#pragma unroll
    for (int u = 0; u < T::NI / 2; ++u)
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            float x[T::MI];
#pragma unroll
            for (int i = 0; i < T::MI; ++i) {
                f32x4 p[2];
                pair_of<T, BCOLS>(acc, i, u, p);
                x[i] = p[h / 4][h % 4];
            }
            f(row, column + 32 * u + h, x);
        }
}

template <class T>
__device__ __forceinline__ Lds16* tile_lds() {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[T::STAGES * T::kStage];
    return (Lds16*)lds;
}

// --- the caller's products ---------------------------------------------------

// N neighbouring values at any element alignment, or those before the row's end.
template <int N>
__device__ __forceinline__ void load_run(const float* p, int left, float (&x)[N]) {
    if (N % 4 == 0 && left >= N) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            const f32x4 v = reinterpret_cast<const f32x4_any*>(p)[k];
            x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = j < left ? p[j] : 0.0f;
}
template <int N>
__device__ __forceinline__ void load_run(const uint16_t* p, int left, float (&x)[N]) {
    if (N == 8 && left >= N) {
        const u32x4 w = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = bf16_to_f32(w[j / 2] >> (16 * (j % 2)) & 0xFFFFu);
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = j < left ? bf16_to_f32(p[j]) : 0.0f;
}
template <int N>
__device__ __forceinline__ void store_run(float* p, const float (&x)[N], int left) {
    if (N % 4 == 0 && left >= N) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k)
            reinterpret_cast<f32x4_any*>(p)[k] = f32x4{x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < left) p[j] = x[j];
}
template <int N>
__device__ __forceinline__ void store_run(uint16_t* p, const float (&x)[N], int left) {
    if (N % 4 == 0 && left >= N) {
        uint32_t w[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
        if constexpr (N == 8) *reinterpret_cast<u32x4_any*>(p) = u32x4{w[0], w[1], w[2], w[3]};
        else if constexpr (N == 4) *reinterpret_cast<u32x2_any*>(p) = u32x2{w[0], w[1]};
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < left) p[j] = (uint16_t)f32_to_bf16_rne(x[j]);
}

// The epilogue of a product: d from alpha times the sums and beta times c.
enum Symmetry : int { kGeneral, kSymmetric, kSymmetricSplit };
template <class T, bool BCOLS, int SYM, typename C, typename D>
__device__ __forceinline__ void product_epilogue(f32x4 (&acc)[T::MI][T::NI], const C* c, D* d, int m, int n, int m0, int n0,
                                                 float alpha, float beta) {
    int row, column;
    lane_place<T>(m0, n0, row, column);
    // of split values the three products are not formed in the same order above the
    // diagonal: a diagonal tile's upper triangle is its lower one's mirror then
    const bool diagonal = SYM != kGeneral && m0 == n0, mirrored = SYM == kSymmetricSplit && diagonal;
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int u = 0; u < T::NI / 2; ++u) {
            const int r = row + i, q = column + 32 * u, left = n - q;
            if (r >= m || left <= 0) continue;
            f32x4 p[2];
            pair_of<T, BCOLS>(acc, i, u, p);
            float x[8] = {p[0].x, p[0].y, p[0].z, p[0].w, p[1].x, p[1].y, p[1].z, p[1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= alpha;
            const int64_t at = (int64_t)r * n + q;
            if (c != nullptr) {
                float y[8];
                load_run(c + at, left, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] += y[j] * beta;
            }
            if (!mirrored) store_run(d + at, x, left);
            if constexpr (SYM != kGeneral) {   // (by rows: not exchanged)
                acc[i][2 * u] = f32x4{x[0], x[1], x[2], x[3]};
                acc[i][2 * u + 1] = f32x4{x[4], x[5], x[6], x[7]};
            }
        }
    if constexpr (SYM != kGeneral) {
        if (diagonal && !mirrored) return;
        each_column<T, BCOLS>(acc, m0, n0, [&](int r, int q, const float (&x)[T::MI]) {
            if (q >= n || r >= m) return;
            if (!mirrored) {
                store_run(d + (int64_t)q * n + r, x, m - r);
                return;
            }
#pragma unroll
            for (int i = 0; i < T::MI; ++i) {
                if (q > r + i || r + i >= m) continue;
                st1(d + (int64_t)(r + i) * n + q, x[i]);
                st1(d + (int64_t)q * n + r + i, x[i]);
            }
        });
    }
}

template <class T, bool BCOLS, int SYM>
__global__ __launch_bounds__(T::kThreads, 2) void products_kernel(const ProductBatch b) {
    uint32_t first;
    const uint32_t w = tile_of<T>(blockIdx.x, gridDim.x);
    const ProductEntry e = b.e[find_tensor(b.tab, (uint32_t)__builtin_amdgcn_readfirstlane((int)w), first)];
    uint32_t ti, tj;
    if constexpr (SYM != kGeneral) tile_in_triangle(w - first, ti, tj);
    else tile_in_bands(w - first, (e.m + T::BM - 1) / T::BM, (e.n + T::BN - 1) / T::BN, ti, tj);
    const Operand a = by_rows(unpack_ptr<const uint16_t>(e.lo[0], e.hi[0]), e.lda, (int)e.m);
    const uint16_t* const right = unpack_ptr<const uint16_t>(e.lo[1], e.hi[0] >> 16);
    const Operand o = BCOLS ? by_columns(right, e.ldb, (int)e.ldb) : by_rows(right, e.ldb, (int)e.n);
    const void* const c = unpack_ptr<const uint16_t>(e.lo[2], e.hi[1]);
    void* const d = unpack_ptr<uint16_t>(e.lo[3], e.hi[1] >> 16);
    const int m0 = (int)ti * T::BM, n0 = (int)tj * T::BN, m = (int)e.m, n = (int)e.n;
    f32x4 acc[T::MI][T::NI];
    multiply<T, true, BCOLS>(a, o, m0, n0, (int)e.k_tiles, tile_lds<T>(), acc);
    auto* const c16 = static_cast<const uint16_t*>(c);
    auto* const c32 = static_cast<const float*>(c);
    auto* const d16 = static_cast<uint16_t*>(d);
    auto* const d32 = static_cast<float*>(d);
    if constexpr (SYM != kGeneral) {   // c is of d's dtype
        if (b.d_bf16) product_epilogue<T, BCOLS, SYM>(acc, c16, d16, m, n, m0, n0, b.alpha, b.beta);
        else product_epilogue<T, BCOLS, SYM>(acc, c32, d32, m, n, m0, n0, b.alpha, b.beta);
    } else if (b.c_bf16) {
        if (b.d_bf16) product_epilogue<T, BCOLS, SYM>(acc, c16, d16, m, n, m0, n0, b.alpha, b.beta);
        else product_epilogue<T, BCOLS, SYM>(acc, c16, d32, m, n, m0, n0, b.alpha, b.beta);
    } else {
        if (b.d_bf16) product_epilogue<T, BCOLS, SYM>(acc, c32, d16, m, n, m0, n0, b.alpha, b.beta);
        else product_epilogue<T, BCOLS, SYM>(acc, c32, d32, m, n, m0, n0, b.alpha, b.beta);
    }
}

// --- the Newton-Schulz steps ---------------------------------------------------

// S = X X^T, or b S + c S S: symmetric, tiles above the diagonal mirrored.
template <class T, bool POLY>
__global__ __launch_bounds__(T::kThreads, 2) void ns_square_kernel(const NsBatch b) {
    uint32_t first, ti, tj;
    const uint32_t w = tile_of<T>(blockIdx.x, gridDim.x);
    const NsEntry e = b.e[find_tensor(b.tab, (uint32_t)__builtin_amdgcn_readfirstlane((int)w), first)];
    tile_in_triangle(w - first, ti, tj);
    const NsPlace p(e.m, e.n);
    char* const base = b.ws + (int64_t)e.base * kNsUnit;
    const int m0 = (int)ti * T::BM, n0 = (int)tj * T::BN, mp = (int)p.mp;
    const int k = POLY ? mp : (int)p.np;
    const uint16_t* const x = reinterpret_cast<const uint16_t*>(base + (POLY ? p.s() : p.hi(b.which)));
    const int across = mp / 64;
    const Operand o = blocked_by_rows(x, k / 64, mp);
    f32x4 acc[T::MI][T::NI];
    multiply<T, false, false>(o, o, m0, n0, k / kTileK, tile_lds<T>(), acc);
    const float cb = b.sc_dev ? b.sc_dev->b : b.b, cc = (b.sc_dev ? b.sc_dev->c : b.c) * (1.0f / kNsScale);
    const _Float16* const s = reinterpret_cast<const _Float16*>(base + p.s());
    _Float16* const out = reinterpret_cast<_Float16*>(base + (POLY ? p.poly() : p.s()));
    int row, column;
    lane_place<T>(m0, n0, row, column);
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int u = 0; u < T::NI / 2; ++u) {
            const bool inside = row + i < mp && column + 32 * u < mp;
            const int64_t at = blocked(min(row + i, mp - 1), min(column + 32 * u, mp - 8), across);
            f16x8 y, h;
            if constexpr (POLY) y = *reinterpret_cast<const f16x8*>(s + at);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float x = acc[i][2 * u + j / 4][j % 4];
                if constexpr (POLY) x = __builtin_fmaf((float)y[j], cb, x * cc);
                else x *= 1.0f / kNsScale;
                acc[i][2 * u + j / 4][j % 4] = x;
                h[j] = (_Float16)x;
            }
            if (inside) *reinterpret_cast<f16x8*>(out + at) = h;
        }
    if (ti == tj) return;
    each_column<T, false>(acc, m0, n0, [&](int r, int q, const float (&x)[T::MI]) {
        if (r >= mp || q >= mp) return;   // both sides are whole runs of 8
        typedef _Float16 Run __attribute__((ext_vector_type(T::MI)));
        Run h;
#pragma unroll
        for (int i = 0; i < T::MI; ++i) h[i] = (_Float16)x[i];
        *reinterpret_cast<Run*>(out + blocked(q, r, across)) = h;
    });
}

// a X + P X (P = b S + c S^2), X's pair as the residual: f(i, u, row, column, x) for
// every eight neighbouring columns inside the padded X, times kNsScale
template <class T, class F>
__device__ __forceinline__ void ns_update(const char* base, const NsPlace& p, int which, float a, int m0, int n0,
                                          f32x4 (&acc)[T::MI][T::NI], F&& f) {
    const int mp = (int)p.mp, np = (int)p.np, across = np / 64;
    const Operand poly = blocked_by_rows(reinterpret_cast<const uint16_t*>(base + p.poly()), mp / 64, mp);
    const Operand x = blocked_by_columns(reinterpret_cast<const uint16_t*>(base + p.hi(which)), across, np);
    multiply<T, false, true>(poly, x, m0, n0, mp / kTileK, tile_lds<T>(), acc);
    const _Float16* const hi = reinterpret_cast<const _Float16*>(base + p.hi(which));
    const _Float16* const lo = reinterpret_cast<const _Float16*>(base + p.lo(which));
    int row, column;
    lane_place<T>(m0, n0, row, column);
    // the loads of ROWS rows before the first use (both column groups of a row: they
    // share its cache line)
    constexpr int kRows = T::MI < kRowsAtOnce ? T::MI : kRowsAtOnce, kU = T::NI / 2;
#pragma unroll
    for (int i0 = 0; i0 < T::MI; i0 += kRows) {
        f16x8 h[kRows][kU], l[kRows][kU];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int64_t at = blocked(min(row + i0 + i, mp - 1), min(column + 32 * u, np - 8), across);
                h[i][u] = *reinterpret_cast<const f16x8*>(hi + at);
                l[i][u] = *reinterpret_cast<const f16x8*>(lo + at);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                f32x4 v[2];
                pair_of<T, true>(acc, i0 + i, u, v);
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = __builtin_fmaf((float)l[i][u][j], a * (1.0f / kNsLow),
                                          __builtin_fmaf((float)h[i][u][j], a, v[j / 4][j % 4] * (1.0f / kNsScale)));
                const int r = row + i0 + i, q = column + 32 * u;
                if (r < mp && q < np) f(i0 + i, u, r, q, y);
            }
    }
}

template <class T>
__global__ __launch_bounds__(T::kThreads, 2) void ns_update_kernel(const NsBatch b) {
    uint32_t first, ti, tj;
    const uint32_t w = tile_of<T>(blockIdx.x, gridDim.x);
    const NsEntry e = b.e[find_tensor(b.tab, (uint32_t)__builtin_amdgcn_readfirstlane((int)w), first)];
    const NsPlace p(e.m, e.n);
    tile_in_bands(w - first, (uint32_t)((p.mp + T::BM - 1) / T::BM), (uint32_t)((p.np + T::BN - 1) / T::BN), ti, tj);
    char* const base = b.ws + (int64_t)e.base * kNsUnit;
    _Float16* const hi = reinterpret_cast<_Float16*>(base + p.hi(1 - b.which));
    _Float16* const lo = reinterpret_cast<_Float16*>(base + p.lo(1 - b.which));
    const int m0 = (int)ti * T::BM, n0 = (int)tj * T::BN;
    f32x4 acc[T::MI][T::NI];
    ns_update<T>(base, p, b.which, b.sc_dev ? b.sc_dev->a : b.a, m0, n0, acc, [&](int, int, int r, int q, const float (&x)[8]) {
        const int64_t at = blocked(r, q, (int)(p.np / 64));
        f16x8 h, l;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            _Float16 y, z;
            split_f16(x[j], y, z);
            h[j] = y;
            l[j] = z;
        }
        *reinterpret_cast<f16x8*>(hi + at) = h;
        *reinterpret_cast<f16x8*>(lo + at) = l;
    });
}

// The epilogue of the last step: X, `scale` times what acc holds, to its destination.
template <int KIND>
struct Destination {
    using P = typename GradType<KIND != kFinalParamF32>::T;
    P* param;
    uint16_t* copy;
    int m, n;
    bool tall;
    float decay, step;
    __device__ __forceinline__ Destination(const FinalEntry& e, const MuonScalars& sc)
        : param(unpack_ptr<P>(e.lo[0], e.hi)), copy(unpack_ptr<uint16_t>(e.lo[1], e.hi >> 16)), m((int)e.m),
          n((int)(e.n & ~kTall)), tall((e.n & kTall) != 0), decay(sc.decay), step(sc.lr * e.scale) {}
    template <int N>
    __device__ __forceinline__ void run(int64_t at, int left, float (&x)[N]) const {
        if constexpr (KIND != kFinalBf16) {
            float p[N];
            load_run(param + at, left, p);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = p[j] * decay - x[j] * step;
        }
        store_run(param + at, x, left);
        if (KIND == kFinalParamF32 && copy != nullptr) store_run(copy + at, x, left);
    }
    // by rows (not tall)
    __device__ __forceinline__ void row(int r, int q, float (&x)[8], float scale) const {
        if (r >= m || q >= n) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= scale;
        run((int64_t)r * n + q, n - q, x);
    }
    // by columns (tall): a column of X is a row of the destination
    template <class T, bool BCOLS>
    __device__ __forceinline__ void columns(const f32x4 (&acc)[T::MI][T::NI], int m0, int n0, float scale) const {
        each_column<T, BCOLS>(acc, m0, n0, [&](int r, int q, float (&x)[T::MI]) {
            if (r >= m || q >= n) return;
#pragma unroll
            for (int i = 0; i < T::MI; ++i) x[i] *= scale;
            run((int64_t)q * m + r, m - r, x);
        });
    }
};

// A norm that is not finite: no step.
template <int KIND>
__device__ __forceinline__ bool skipped(const FinalBatch& b, const MuonScalars& sc) {
    if constexpr (KIND == kFinalBf16) return false;
    return b.norm_sq != nullptr && !__builtin_isfinite(*b.norm_sq + sc.extra_norm_sq);
}

template <class T, int KIND>
__global__ __launch_bounds__(T::kThreads, 2) void ns_final_kernel(const FinalBatch b) {
    uint32_t first, ti, tj;
    const uint32_t w = tile_of<T>(blockIdx.x, gridDim.x);
    const FinalEntry e = b.e[find_tensor(b.tab, (uint32_t)__builtin_amdgcn_readfirstlane((int)w), first)];
    const MuonScalars& sc = b.sc_dev ? *b.sc_dev : b.sc;
    if (skipped<KIND>(b, sc)) return;
    const Destination<KIND> to(e, sc);
    const NsPlace p(to.m, to.n);
    tile_in_bands(w - first, (uint32_t)((to.m + T::BM - 1) / T::BM), (uint32_t)((to.n + T::BN - 1) / T::BN), ti, tj);
    const int m0 = (int)ti * T::BM, n0 = (int)tj * T::BN;
    f32x4 acc[T::MI][T::NI];
    const char* const base = b.ws + (int64_t)e.base * kNsUnit;
    if (!to.tall) {
        ns_update<T>(base, p, b.which, sc.a, m0, n0, acc,
                     [&](int, int, int r, int q, float (&x)[8]) { to.row(r, q, x, 1.0f / kNsScale); });
    } else {
        ns_update<T>(base, p, b.which, sc.a, m0, n0, acc, [&](int i, int u, int, int, const float (&x)[8]) {
            acc[i][2 * u] = f32x4{x[0], x[1], x[2], x[3]};
            acc[i][2 * u + 1] = f32x4{x[4], x[5], x[6], x[7]};
        });
        to.template columns<T, false>(acc, m0, n0, 1.0f / kNsScale);
    }
}

// --- matrices whose short side is at most 64 -------------------------------------

// Columns [n0, n0 + 64) of Q X, in units of skinny_scale.
__device__ __forceinline__ void skinny_product(const char* base, const SkinnyPlace& p, int n0, f32x4 (&acc)[T64::MI][T64::NI]) {
    const Operand q = by_rows(reinterpret_cast<const uint16_t*>(base + p.q()), 3 * kSkinny, (int)kSkinny);
    const Operand x = blocked_by_columns(reinterpret_cast<const uint16_t*>(base), (int)(p.np / 64), (int)p.np);
    multiply<T64, false, true>(q, x, 0, n0, 3, tile_lds<T64>(), acc);
}
__device__ __forceinline__ float skinny_scale(const char* base, const SkinnyPlace& p) {
    return *reinterpret_cast<const float*>(base + p.scale());
}

// One partial sum of S from the pairs: hi hi^T + hi lo^T + lo hi^T (the fourth
// product is below fp32's last bit).  APPLY: of Q X, which takes X's place: a workgroup
// reads and writes its own columns alone, 64 at a time, all of them in LDS before the
// first is written.
template <bool APPLY>
__global__ __launch_bounds__(T64::kThreads, 2) void skinny_gram_kernel(const NsBatch b) {
    uint32_t first;
    const NsEntry e = b.e[find_tensor(b.tab, blockIdx.x, first)];
    const SkinnyPlace p(e.n);
    char* const base = b.ws + (int64_t)e.base * kNsUnit;
    const int64_t chunk = blockIdx.x - first, from = chunk * p.chunk, left = p.np / kTileK - from;
    const int tiles = (int)(left < p.chunk ? left : p.chunk);
    const int across = (int)(p.np / 64);
    if constexpr (APPLY) {
        const float scale = skinny_scale(base, p) * kNsScale;
        _Float16* const x0 = reinterpret_cast<_Float16*>(base);
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int n0 = (int)(from + t) * T64::BN;
            f32x4 acc[T64::MI][T64::NI];
            skinny_product(base, p, n0, acc);
            each_row<T64, true>(acc, 0, n0, [&](int r, int c, const float (&x)[8]) {
                const int64_t at = blocked(r, c, across);
                f16x8 h, l;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    _Float16 y, z;
                    split_f16(x[j] * scale, y, z);
                    h[j] = y;
                    l[j] = z;
                }
                *reinterpret_cast<f16x8*>(x0 + at) = h;
                *reinterpret_cast<f16x8*>(x0 + p.x / 2 + at) = l;
                *reinterpret_cast<f16x8*>(x0 + p.x + at) = h;
            });
        }
        // what the other waves stored is read below
        loads_done<0>();
        __threadfence_block();
        __syncthreads();
    }
    const uint16_t* const x = reinterpret_cast<const uint16_t*>(base) + from * kBlockElems;
    const Operand hi = blocked_by_rows(x, across, (int)kSkinny), lo = blocked_by_rows(x + p.x / 2, across, (int)kSkinny);
    f32x4 sum[T64::MI][T64::NI], acc[T64::MI][T64::NI];
    multiply<T64, false, false>(hi, lo, 0, 0, tiles, tile_lds<T64>(), sum);
    multiply<T64, false, false>(lo, hi, 0, 0, tiles, tile_lds<T64>(), acc);
#pragma unroll
    for (int i = 0; i < T64::MI; ++i)
#pragma unroll
        for (int j = 0; j < T64::NI; ++j) sum[i][j] = (sum[i][j] + acc[i][j]) * (1.0f / kNsLow);
    multiply<T64, false, false>(hi, hi, 0, 0, tiles, tile_lds<T64>(), acc);
    float* const out = reinterpret_cast<float*>(base + p.parts() + chunk * SkinnyPlace::kPart);
#pragma unroll
    for (int i = 0; i < T64::MI; ++i)
#pragma unroll
        for (int j = 0; j < T64::NI; ++j) acc[i][j] += sum[i][j];
    each_row<T64, false>(acc, 0, 0, [&](int r, int q, const float (&x)[8]) { store_run(out + r * kSkinny + q, x, 8); });
}

// 64 x 64 matrices in LDS, rows of 65 words.
constexpr int kPitch = 65;
struct Square {
    float v[kSkinny * kPitch];
};

// f(row, column, value) of x y: each of 16 waves forms 16 x 16 with the fp32 matrix
// instruction (lane l: row l % 16 of a and column l % 16 of b at k = l / 16).  One
// matrix's products follow one another, so that their latency counts: with 4 waves
// of 16 x 64 each the kernel took 39 us (25 so).
constexpr int kStepThreads = 1024;
template <class F>
__device__ __forceinline__ void square_product(const Square& x, const Square& y, F&& f) {
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, row = wave / 4 * 16, col = wave % 4 * 16, at = l & 15, kl = l >> 4;
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int k = 0; k < kSkinny; k += 8)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            acc[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.v[(row + at) * kPitch + k + 4 * h + kl],
                                                          y.v[(k + 4 * h + kl) * kPitch + col + at], acc[h], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) f(row + 4 * kl + i, col + at, acc[0][i] + acc[1][i]);
}

// acc += y y^T, as square_product forms it.
__device__ __forceinline__ void add_square(const Square& y, f32x4 (&acc)[2]) {
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, row = wave / 4 * 16, col = wave % 4 * 16, at = l & 15, kl = l >> 4;
#pragma unroll
    for (int k = 0; k < kSkinny; k += 8)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            acc[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(y.v[(row + at) * kPitch + k + 4 * h + kl],
                                                          y.v[(col + at) * kPitch + k + 4 * h + kl], acc[h], 0, 0, 0);
}
// f(row, column) of this lane's four results of those
template <class F>
__device__ __forceinline__ void each_result(F&& f) {
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 4; ++i) f(i, wave / 4 * 16 + 4 * (l >> 4) + i, wave % 4 * 16 + (l & 15));
}

// Q = M_1 M_2 ... of `steps` steps with M = a I + b S + c S^2 and S <- M S M after each
// (all polynomials of the first S: they commute).  I has the matrix's own rows
// alone: a^steps in the padding would be most of Q's largest value, to which its scale
// goes (3.4445^20 = 5e10), and leave its other values few bits or none.
__device__ __forceinline__ void polynomials(Square& s, Square& t, Square& m, Square& q, int rows, int steps, float ca, float cb,
                                            float cc) {
    for (int step = 0; step < steps; ++step) {
        square_product(s, s, [&](int r, int c, float x) {
            const int at = r * kPitch + c;
            m.v[at] = (s.v[at] * cb + x * cc) + (r == c && r < rows ? ca : 0.0f);
            if (step == 0) q.v[at] = m.v[at];
        });
        __syncthreads();
        const bool more = step + 1 < steps;
        if (step > 0) {
            // q's own product: kept until every wave has read q
            f32x4 kept;
            int n = 0;
            square_product(m, q, [&](int, int, float x) { kept[n++] = x; });
            __syncthreads();
            each_result([&](int i, int r, int c) { q.v[r * kPitch + c] = kept[i]; });
        }
        if (more) {
            square_product(m, s, [&](int r, int c, float x) { t.v[r * kPitch + c] = x; });
            __syncthreads();
            square_product(t, m, [&](int r, int c, float x) { s.v[r * kPitch + c] = x; });
        }
        __syncthreads();
    }
}

// X <- Q X and S anew, by one workgroup: 64 columns at a time in LDS, every
// thread the same four elements of them.  There may be 2^20 columns: the sums of every
// 1024 are added in binary64.
__device__ __forceinline__ void apply_alone(char* base, const SkinnyPlace& p, const Square& q, Square& s, Square& t, Square& m) {
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    const int own = threadIdx.x * 4, place = own / (int)kSkinny * kPitch + own % (int)kSkinny;
    const int blocks = (int)(p.np / kSkinny);
    double total[4] = {0.0, 0.0, 0.0, 0.0};
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll 1
    for (int k = 0; k < blocks; ++k) {
        _Float16* const hi = reinterpret_cast<_Float16*>(base) + (int64_t)k * kBlockElems + own;
        _Float16 *const lo = hi + p.x / 2, *const again = hi + p.x;
        f16x4 h = *reinterpret_cast<const f16x4*>(hi), l = *reinterpret_cast<const f16x4*>(lo);
#pragma unroll
        for (int j = 0; j < 4; ++j) t.v[place + j] = __builtin_fmaf((float)l[j], 1.0f / kNsLow, (float)h[j]);
        __syncthreads();
        square_product(q, t, [&](int r, int c, float x) { m.v[r * kPitch + c] = x; });
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            _Float16 y, z;
            split_f16(m.v[place + j], y, z);
            h[j] = y;
            l[j] = z;
            m.v[place + j] = __builtin_fmaf((float)z, 1.0f / kNsLow, (float)y);
        }
        *reinterpret_cast<f16x4*>(hi) = h;
        *reinterpret_cast<f16x4*>(lo) = l;
        *reinterpret_cast<f16x4*>(again) = h;
        __syncthreads();
        add_square(m, acc);   // (the next m is written two barriers on)
        if (k % 16 == 15 || k + 1 == blocks) {
#pragma unroll
            for (int i = 0; i < 4; ++i) total[i] += (double)acc[0][i] + (double)acc[1][i];
            acc[0] = acc[1] = f32x4{0, 0, 0, 0};
        }
    }
    each_result([&](int i, int r, int c) { s.v[r * kPitch + c] = (float)(total[i] * (1.0 / (kNsScale * kNsScale))); });
    __syncthreads();
}

// The product Q of b.steps steps' polynomials, as two fp16 values times a power of two, in
// the form of Q X's left operand: [hi | hi / kNsLow | lo].  Where they are too many for
// one product (kSkinnyGrowth), of the last ones, X having become what the others make of it.
__global__ __launch_bounds__(kStepThreads) void skinny_steps_kernel(const NsBatch b) {
    __shared__ Square s, t, m, q;
    const NsEntry e = b.e[blockIdx.x];
    const SkinnyPlace p(e.n);
    char* const base = b.ws + (int64_t)e.base * kNsUnit;
    const float ca = b.sc_dev ? b.sc_dev->a : b.a, cb = b.sc_dev ? b.sc_dev->b : b.b, cc = b.sc_dev ? b.sc_dev->c : b.c;
    const float* const parts = reinterpret_cast<const float*>(base + p.parts());
    for (int i = threadIdx.x; i < kSkinny * kSkinny; i += kStepThreads) {
        float x = 0.0f;
        for (int64_t k = 0; k < p.chunks; ++k) x += parts[k * (kSkinny * kSkinny) + i];
        s.v[i / kSkinny * kPitch + i % kSkinny] = x * (1.0f / (kNsScale * kNsScale));
    }
    __syncthreads();
    const int at_once = skinny_steps_at_once(ca);
    int left = b.steps;
    for (; left > at_once; left -= at_once) {
        polynomials(s, t, m, q, (int)e.m, at_once, ca, cb, cc);
        apply_alone(base, p, q, s, t, m);
    }
    polynomials(s, t, m, q, (int)e.m, left, ca, cb, cc);
    // the scale: Q's largest magnitude to [2^12, 2^13), by a power of two that binary32 has
    // (2^127 at most: a Q below 2^-115 stays smaller)
    float most = 0.0f;
    for (int i = threadIdx.x; i < kSkinny * kSkinny; i += kStepThreads)
        most = fmaxf(most, fabsf(q.v[i / kSkinny * kPitch + i % kSkinny]));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) t.v[threadIdx.x >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kStepThreads / 64; ++w) most = fmaxf(most, t.v[w]);
    int exponent = 0;
    if (most > 0.0f && __builtin_isfinite(most)) (void)frexpf(most, &exponent);
    exponent = max(exponent, 13 - 127);
    const float scale = ldexpf(1.0f, 13 - exponent);
    _Float16* const out = reinterpret_cast<_Float16*>(base + p.q());
    for (int i = threadIdx.x; i < kSkinny * kSkinny; i += kStepThreads) {
        const int r = i / (int)kSkinny, c = i % (int)kSkinny;
        const float x = q.v[r * kPitch + c] * scale;
        _Float16 h, l;
        split_f16(x, h, l);
        out[r * 3 * kSkinny + c] = h;
        out[r * 3 * kSkinny + kSkinny + c] = (_Float16)((float)h * (1.0f / kNsLow));
        out[r * 3 * kSkinny + 2 * kSkinny + c] = (_Float16)((float)l * (1.0f / kNsLow));
    }
    if (threadIdx.x == 0) *reinterpret_cast<float*>(base + p.scale()) = ldexpf(1.0f / kNsScale, exponent - 13);
}

template <int KIND>
__global__ __launch_bounds__(T64::kThreads, 2) void skinny_final_kernel(const FinalBatch b) {
    uint32_t first;
    const FinalEntry e = b.e[find_tensor(b.tab, blockIdx.x, first)];
    const MuonScalars& sc = b.sc_dev ? *b.sc_dev : b.sc;
    if (skipped<KIND>(b, sc)) return;
    const Destination<KIND> to(e, sc);
    const SkinnyPlace p(to.n);
    const char* const base = b.ws + (int64_t)e.base * kNsUnit;
    const int n0 = (int)(blockIdx.x - first) * T64::BN;
    f32x4 acc[T64::MI][T64::NI];
    skinny_product(base, p, n0, acc);
    const float scale = skinny_scale(base, p);
    if (to.tall) to.template columns<T64, true>(acc, 0, n0, scale);
    else each_row<T64, true>(acc, 0, n0, [&](int r, int c, float (&x)[8]) { to.row(r, c, x, scale); });
}

template <class T>
void launch_products_of(const ProductBatch& b, bool b_cols, bool sym, bool split, unsigned tiles, hipStream_t stream) {
    const dim3 grid(tiles), block(T::kThreads);
    if (sym && split) hipLaunchKernelGGL((products_kernel<T, false, kSymmetricSplit>), grid, block, 0, stream, b);
    else if (sym) hipLaunchKernelGGL((products_kernel<T, false, kSymmetric>), grid, block, 0, stream, b);
    else if (b_cols) hipLaunchKernelGGL((products_kernel<T, true, kGeneral>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((products_kernel<T, false, kGeneral>), grid, block, 0, stream, b);
}

template <class T>
void launch_ns_of(const NsBatch& b, int phase, unsigned tiles, hipStream_t stream) {
    const dim3 grid(tiles), block(T::kThreads);
    if (phase == kNsGram) hipLaunchKernelGGL((ns_square_kernel<T, false>), grid, block, 0, stream, b);
    else if (phase == kNsPoly) hipLaunchKernelGGL((ns_square_kernel<T, true>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((ns_update_kernel<T>), grid, block, 0, stream, b);
}

template <class T>
void launch_final_of(const FinalBatch& b, int kind, unsigned tiles, hipStream_t stream) {
    const dim3 grid(tiles), block(T::kThreads);
    if (kind == kFinalBf16) hipLaunchKernelGGL((ns_final_kernel<T, kFinalBf16>), grid, block, 0, stream, b);
    else if (kind == kFinalParamF32) hipLaunchKernelGGL((ns_final_kernel<T, kFinalParamF32>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((ns_final_kernel<T, kFinalParamBf16>), grid, block, 0, stream, b);
}

}  // namespace

hipError_t launch_products(const ProductBatch& b, int size, bool b_cols, bool sym, bool split, int64_t tiles,
                           hipStream_t stream) {
    if (size == kTile256) launch_products_of<T256>(b, b_cols, sym, split, (unsigned)tiles, stream);
    else if (size == kTile128) launch_products_of<T128>(b, b_cols, sym, split, (unsigned)tiles, stream);
    else launch_products_of<T64>(b, b_cols, sym, split, (unsigned)tiles, stream);
    return hipGetLastError();
}

hipError_t launch_ns(const NsBatch& b, int phase, int size, int64_t tiles, hipStream_t stream) {
    if (size == kTile256) launch_ns_of<T256>(b, phase, (unsigned)tiles, stream);
    else if (size == kTile128) launch_ns_of<T128>(b, phase, (unsigned)tiles, stream);
    else launch_ns_of<T64>(b, phase, (unsigned)tiles, stream);
    return hipGetLastError();
}

hipError_t launch_skinny_gram(const NsBatch& b, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(T64::kThreads);
    if (b.which) hipLaunchKernelGGL((skinny_gram_kernel<true>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((skinny_gram_kernel<false>), grid, block, 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_skinny_steps(const NsBatch& b, int64_t count, hipStream_t stream) {
    hipLaunchKernelGGL(skinny_steps_kernel, dim3((unsigned)count), dim3(kStepThreads), 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_ns_final(const FinalBatch& b, int kind, int size, bool skinny, int64_t tiles, hipStream_t stream) {
    if (skinny) {
        const dim3 grid((unsigned)tiles), block(T64::kThreads);
        if (kind == kFinalBf16) hipLaunchKernelGGL((skinny_final_kernel<kFinalBf16>), grid, block, 0, stream, b);
        else if (kind == kFinalParamF32) hipLaunchKernelGGL((skinny_final_kernel<kFinalParamF32>), grid, block, 0, stream, b);
        else hipLaunchKernelGGL((skinny_final_kernel<kFinalParamBf16>), grid, block, 0, stream, b);
        return hipGetLastError();
    }
    if (size == kTile256) launch_final_of<T256>(b, kind, (unsigned)tiles, stream);
    else if (size == kTile128) launch_final_of<T128>(b, kind, (unsigned)tiles, stream);
    else launch_final_of<T64>(b, kind, (unsigned)tiles, stream);
    return hipGetLastError();
}

}  // namespace zs
