// C-ABI entry points over lists of matrices (include/zshard_matrices.h):
// validation on the host, then launches of as many matrices as their tables hold.
#include <cstddef>

#include "../../include/zshard_matrices.h"
#include "lists.h"
#include "matrices.h"

using namespace zs;

static_assert(sizeof(zs_muon_scalars) == sizeof(MuonScalars) && offsetof(zs_muon_scalars, eps) == offsetof(MuonScalars, eps) &&
                  offsetof(zs_muon_scalars, nesterov) == offsetof(MuonScalars, nesterov), "scalar layout");

namespace {

constexpr int64_t kMaxElemsOfMatrix = (int64_t(1) << 31) - 1;
constexpr uintptr_t kWorkspaceAlign = 256;

bool sides_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 0 && rows <= ZS_MATRIX_MAX_SIDE && cols <= ZS_MATRIX_MAX_SIDE &&
           rows * cols <= kMaxElemsOfMatrix;
}

// The tile that launches of a list use, from how many of each size one of them has
// (a table of `most` matrices to a launch): the largest one of which there are
// enough.  Larger tiles read their operands less often, so where a tile is long in k
// 192 of them (on 256 CUs) are enough; short ones are mostly their first loads and their
// epilogue, of which smaller tiles have several to a CU at a time.  224 matrices of 251
// x 683, k up to 683, 64 / 128 / 192 / 256 / 512 enough: gram 162 / 98 / 98 / 92 / 92 us, muon step 684 /
// 685 / 684 / 684 / 632; 4096 x 4096 x 4096 (256 tiles of 256 x 256, 1024 of 128 x 128): 1221 and 1046 TFLOP/s.
struct TileCount {
    int64_t of[3] = {0, 0, 0};
    int64_t matrices = 0, longest = 0;
    void add(int64_t rows, int64_t cols, int64_t k, bool triangle) {
        for (int s = 0; s < 3; ++s) {
            const int64_t r = ceil_div(rows, tile_side(s));
            of[s] += triangle ? r * (r + 1) / 2 : r * ceil_div(cols, tile_side(s));
        }
        ++matrices;
        longest = std::max(longest, k);
    }
    int size(int64_t most) const {
        const int64_t launches = ceil_div(std::max(matrices, (int64_t)1), most);
        const int64_t enough = (longest >= 1024 ? 192 : 512) * launches;
        return of[kTile256] >= enough ? kTile256 : of[kTile128] >= enough ? kTile128 : kTile64;
    }
};

// Checks that every call shares: the list, and the workspace against `need`.
int32_t check_workspace(const void* ws, int64_t bytes, int64_t need) {
    if (need > 0 && (ws == nullptr || !aligned(ws, kWorkspaceAlign))) return ZS_EINVAL;
    return bytes < need ? ZS_EWORKSPACE : ZS_OK;
}
bool typed(const void* p, int32_t dtype) { return p != nullptr && aligned(p, (uintptr_t)elem_size(dtype)) && packable(p); }

// --- products ------------------------------------------------------------------

// One operand of a product: where the kernels find it, and what it needs of the
// workspace to be there.
struct Side {
    bool direct;
    int64_t bytes;   // of one copy in the workspace
};
// rows x k with k innermost, or (columns form) k x rows
Side side_of(const void* p, int32_t dtype, int64_t rows, int64_t k, bool columns, bool transposed) {
    Side s;
    s.direct = dtype == ZS_BF16 && !transposed && k % kPadSide == 0 && aligned(p, 16) && (!columns || rows % 8 == 0);
    s.bytes = s.direct ? 0 : pad_side(rows) * pad_side(k) * 2 * (dtype == ZS_BF16 ? 1 : 3);
    return s;
}

// One product in either call's terms
struct Product {
    const void *a, *b, *c;
    void* d;
    int64_t m, n, k;
    bool a_transposed, b_transposed;   // a^T is k x m in memory; the columns form of b is k x n
    bool gram;
};
Product product_of(const zs_product& p, int32_t flags) {
    return Product{p.a, p.b, p.c, p.d, p.m, p.n, p.k, (flags & ZS_TRANSPOSE_A) != 0, (flags & ZS_TRANSPOSE_B) != 0, false};
}
Product product_of(const zs_gram& p, int32_t) {
    const int64_t m = p.transposed ? p.cols : p.rows, k = p.transposed ? p.rows : p.cols;
    return Product{p.a, p.a, p.c, p.d, m, m, k, p.transposed != 0, true, true};
}
bool shape_ok(const zs_product& p) { return sides_ok(p.m, p.n) && sides_ok(p.m, p.k) && sides_ok(p.k, p.n); }
bool shape_ok(const zs_gram& p) {
    const int64_t m = p.transposed ? p.cols : p.rows;
    return sides_ok(p.rows, p.cols) && sides_ok(m, m) && (p.transposed == 0 || p.transposed == 1) && p.reserved == 0;
}

// Places of one product's operands in the workspace, from `at` on.
struct Placed {
    Side a, b;
    int64_t a_at, b_at, end;
    bool shared;     // b is a's copy
};
Placed place(const Product& p, int32_t dtype, int64_t at) {
    Placed q;
    q.a = side_of(p.a, dtype, p.m, p.k, false, p.a_transposed);
    // a gram of bf16 values reads one copy twice
    const bool one = q.shared = p.gram && dtype == ZS_BF16;
    q.b = one ? q.a : side_of(p.b, dtype, p.n, p.k, !p.b_transposed, p.gram && p.a_transposed);
    q.a_at = at;
    at += ceil_div(q.a.bytes, 256) * 256;
    q.b_at = one ? q.a_at : at;
    if (!one) at += ceil_div(q.b.bytes, 256) * 256;
    q.end = at;
    return q;
}

template <typename T>
int64_t products_workspace(const T* list, int32_t count, int32_t in_dtype, int32_t flags) {
    if (count < 0 || (count > 0 && list == nullptr) || !dtype_ok(in_dtype)) return -1;
    int64_t at = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (!shape_ok(list[k])) return -1;
        const Product p = product_of(list[k], flags);
        if (p.m == 0 || p.n == 0 || p.k == 0) continue;
        at = place(p, in_dtype, at).end;
        if (at > kMaxElems * 8) return -1;
    }
    return at;
}

template <typename T>
int32_t products(const T* list, int32_t count, int32_t in_dtype, int32_t c_dtype, int32_t d_dtype, int32_t flags,
                 double alpha, double beta, void* workspace, int64_t workspace_bytes, void* hip_stream) {
    const int64_t need = products_workspace(list, count, in_dtype, flags);
    if (need < 0 || !dtype_ok(c_dtype) || !dtype_ok(d_dtype)) return ZS_EINVAL;
    if (!finite_float(alpha) || !finite_float(beta)) return ZS_EINVAL;
    int32_t rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != ZS_OK) return rc;
    Ranges ranges;
    if (!ranges.reserve(count, 5)) return ZS_EINVAL;
    TileCount tiles;
    const int64_t isz = elem_size(in_dtype);
    for (int32_t k = 0; k < count; ++k) {
        const Product p = product_of(list[k], flags);
        if (p.m == 0 || p.n == 0) continue;
        if (!typed(p.d, d_dtype)) return ZS_EINVAL;
        if (p.k > 0 && (!typed(p.a, in_dtype) || !typed(p.b, in_dtype))) return ZS_EINVAL;
        if (p.c != nullptr && !typed(p.c, c_dtype)) return ZS_EINVAL;
        ranges.add(0, p.a, p.m * p.k * isz, false);
        if (!p.gram) ranges.add(1, p.b, p.k * p.n * isz, false);
        if (!(p.c == p.d && c_dtype == d_dtype)) ranges.add(2, p.c, p.m * p.n * elem_size(c_dtype), false);
        ranges.add(3, p.d, p.m * p.n * elem_size(d_dtype), true);
        tiles.add(p.m, p.n, p.k, p.gram);
    }
    if (count > 0) ranges.add(4, workspace, need, true);
    if (ranges.clash()) return ZS_EOVERLAP;

    char* const ws = static_cast<char*>(workspace);
    const bool b_cols = !std::is_same<T, zs_gram>::value && (flags & ZS_TRANSPOSE_B) == 0;
    // copies: first all a, then all b (each kind of copy is a launch of its own)
    for (int side = 0; side < 2; ++side)
        for (int transposed = 0; transposed < 2; ++transposed) {
            StageBatch s;
            std::memset(&s, 0, sizeof(s));
            const bool columns = side == 1 && b_cols;
            const int kind = in_dtype == ZS_BF16 ? kStagePlain : side == 0 ? kStageHiHiLo : kStageHiLoHi;
            auto launch = [&](const StageBatch& x, int64_t n) {
                return launch_stage(x, in_dtype == ZS_BF16, kind, columns, transposed != 0, n, as_stream(hip_stream));
            };
            Filler<StageBatch, decltype(launch)> fill(s, launch);
            int64_t at = 0;
            for (int32_t k = 0; k < count; ++k) {
                const Product p = product_of(list[k], flags);
                if (p.m == 0 || p.n == 0 || p.k == 0) continue;
                const Placed q = place(p, in_dtype, at);
                at = q.end;
                const Side& o = side == 0 ? q.a : q.b;
                if (o.direct || (side == 1 && q.shared)) continue;
                const bool turned = p.gram || side == 0 ? p.a_transposed : false;
                if (turned != (transposed != 0)) continue;
                const int64_t rows = columns ? p.k : side == 0 ? p.m : p.n, cols = columns ? p.n : p.k;
                int e = 0;
                rc = fill.add(stage_tiles(rows, cols), e);
                if (rc != ZS_OK) return rc;
                const void* const src = side == 0 ? p.a : p.b;
                const void* const dst = ws + (side == 0 ? q.a_at : q.b_at);
                s.e[e] = StageEntry{{ptr_lo(src), ptr_lo(dst)}, ptr_hi(src) | ptr_hi(dst) << 16, (uint32_t)rows, (uint32_t)cols};
            }
            rc = fill.flush();
            if (rc != ZS_OK) return rc;
        }

    ProductBatch b;
    std::memset(&b, 0, sizeof(b));
    b.alpha = (float)alpha;
    b.beta = (float)beta;
    b.c_bf16 = c_dtype == ZS_BF16;
    b.d_bf16 = d_dtype == ZS_BF16;
    const int size = tiles.size(sizeof(b.e) / sizeof(b.e[0]));
    constexpr bool kGram = std::is_same<T, zs_gram>::value;
    auto launch = [&](const ProductBatch& x, int64_t n) {
        return launch_products(x, size, b_cols, kGram, in_dtype != ZS_BF16, n, as_stream(hip_stream));
    };
    Filler<ProductBatch, decltype(launch)> fill(b, launch);
    int64_t at = 0;
    for (int32_t k = 0; k < count; ++k) {
        const Product p = product_of(list[k], flags);
        if (p.m == 0 || p.n == 0) continue;
        const int parts = in_dtype == ZS_BF16 ? 1 : 3;
        const void *a = p.a, *o = p.b, *c = b.beta == 0.0f ? nullptr : p.c;
        int64_t lda = p.k, ldb = b_cols ? p.n : p.k, kp = p.k;
        if (p.k > 0) {
            const Placed q = place(p, in_dtype, at);
            at = q.end;
            kp = pad_side(p.k) * parts;
            if (!q.a.direct) a = ws + q.a_at, lda = kp;
            if (!q.b.direct) o = ws + q.b_at, ldb = b_cols ? pad_side(p.n) : kp;
        }
        TileCount one;
        one.add(p.m, p.n, p.k, kGram);
        int e = 0;
        rc = fill.add(one.of[size], e);
        if (rc != ZS_OK) return rc;
        b.e[e] = ProductEntry{{ptr_lo(a), ptr_lo(o), ptr_lo(c), ptr_lo(p.d)},
                              {ptr_hi(a) | ptr_hi(o) << 16, ptr_hi(c) | ptr_hi(p.d) << 16},
                              (uint32_t)p.m, (uint32_t)p.n, (uint32_t)(kp / kPadSide), (uint32_t)lda, (uint32_t)ldb};
    }
    return fill.flush();
}

// --- Newton-Schulz steps -----------------------------------------------------------

// One matrix in either call's terms
struct Matrix {
    const void* in;      // gradient, or input
    float* momentum;
    void* out;           // parameter, or output
    uint16_t* copy;
    int64_t rows, cols;
    float scale;
    int64_t m() const { return std::min(rows, cols); }
    int64_t n() const { return std::max(rows, cols); }
    uint32_t n_tall() const { return (uint32_t)n() | (rows > cols ? kTall : 0u); }
};
Matrix matrix_of(const zs_muon_matrix& x) {
    return Matrix{x.grad, x.momentum, x.param, x.param_bf16, x.rows, x.cols, (float)x.scale};
}
Matrix matrix_of(const zs_orthogonal& x) { return Matrix{x.in, nullptr, x.out, nullptr, x.rows, x.cols, 1.0f}; }

// A list is worked through in groups of consecutive matrices that share the
// workspace: as many as kGroupElems elements hold, one at least.
constexpr int64_t kGroupElems = int64_t(1) << 29;
struct Group {
    int32_t first, last;      // [first, last)
    int64_t units;            // of kNsUnit
    int64_t partials;
    int64_t partials_at() const { return units * kNsUnit; }
    int64_t inverse_at() const { return partials_at() + partials * 8; }
    // f(matrix, its place in kNsUnit) for each matrix that has elements
    template <typename T, typename F>
    int32_t each(const T* list, F&& f) const;
    int64_t bytes() const { return inverse_at() + (int64_t)(last - first) * 4; }
};
template <typename T, typename F>
int32_t Group::each(const T* list, F&& f) const {
    int64_t unit = 0;
    for (int32_t k = first; k < last; ++k) {
        const Matrix x = matrix_of(list[k]);
        if (x.rows == 0 || x.cols == 0) continue;
        const int32_t rc = f(x, unit);
        if (rc != ZS_OK) return rc;
        unit += ns_bytes(x.m(), x.n()) / kNsUnit;
    }
    return ZS_OK;
}
template <typename T>
Group group_from(const T* list, int32_t count, int32_t first) {
    Group g = {first, first, 0, 0};
    int64_t elems = 0;
    for (; g.last < count; ++g.last) {
        const Matrix x = matrix_of(list[g.last]);
        if (x.rows == 0 || x.cols == 0) continue;
        const int64_t n = pad_side(x.rows) * pad_side(x.cols);
        if (elems > 0 && elems + n > kGroupElems) break;
        elems += n;
        g.units += ns_bytes(x.m(), x.n()) / kNsUnit;
        g.partials += ceil_div(x.rows * x.cols, kMomentumTile);
    }
    return g;
}

template <typename T>
int64_t ns_workspace(const T* list, int32_t count) {
    if (count < 0 || (count > 0 && list == nullptr)) return -1;
    for (int32_t k = 0; k < count; ++k)
        if (!sides_ok(list[k].rows, list[k].cols)) return -1;
    int64_t need = 0;
    for (int32_t k = 0; k < count;) {
        const Group g = group_from(list, count, k);
        if (g.partials > 0) need = std::max(need, ceil_div(g.bytes(), 256) * 256);
        k = g.last;
    }
    return need;
}

bool coefficient_ok(double x) { return std::fabs(x) <= 32.0; }
bool eps_ok(double x) { return x >= 1e-30 && std::isfinite(x); }

template <typename T>
int32_t run_ns(const T* list, int32_t count, int32_t in_dtype, int kind, int32_t steps, const MuonScalars& sc,
               const MuonScalars* sc_dev, const double* norm_sq, char* ws, void* hip_stream) {
    const hipStream_t stream = as_stream(hip_stream);
    const bool momentum = kind != kFinalBf16;
    int32_t rc;
    for (int32_t from = 0; from < count;) {
        const Group g = group_from(list, count, from);
        from = g.last;
        if (g.partials == 0) continue;
        double* const partials = reinterpret_cast<double*>(ws + g.partials_at());
        float* const inverse = reinterpret_cast<float*>(ws + g.inverse_at());

        // new momentum, sums of squares
        {
            MomentumBatch b;
            std::memset(&b, 0, sizeof(b));
            b.sc = sc;
            b.sc_dev = sc_dev;
            b.norm_sq = norm_sq;
            b.partials = partials;
            auto launch = [&](MomentumBatch& x, int64_t tiles) {
                const hipError_t e = launch_momentum(x, in_dtype == ZS_BF16, momentum, tiles, stream);
                x.partials += tiles;
                return e;
            };
            Filler<MomentumBatch, decltype(launch)> fill(b, launch);
            rc = g.each(list, [&](const Matrix& x, int64_t) -> int32_t {
                int e = 0;
                const int32_t failed = fill.add(ceil_div(x.rows * x.cols, kMomentumTile), e);
                if (failed != ZS_OK) return failed;
                b.e[e] = MomentumEntry{{ptr_lo(x.in), ptr_lo(x.momentum)}, ptr_hi(x.in) | ptr_hi(x.momentum) << 16,
                                       (uint32_t)(x.rows * x.cols)};
                return ZS_OK;
            });
            if (rc != ZS_OK) return rc;
            rc = fill.flush();
            if (rc != ZS_OK) return rc;
        }
        int64_t most_partials = 0;
        g.each(list, [&](const Matrix& x, int64_t) {
            most_partials = std::max(most_partials, ceil_div(x.rows * x.cols, kMomentumTile));
            return ZS_OK;
        });
        if (most_partials > kPackPartials) {
            NormsBatch b;
            std::memset(&b, 0, sizeof(b));
            b.partials = partials;
            b.sc_dev = sc_dev;
            b.eps = sc.eps;
            constexpr uint32_t kMost = sizeof(b.start) / sizeof(b.start[0]) - 1;
            int64_t at = 0;
            uint32_t done = 0;
            auto launch = [&]() -> int32_t {
                if (b.count == 0) return ZS_OK;
                b.inverse = inverse + done;
                done += b.count;
                const int32_t r = hip_status(launch_inverse_norms(b, stream));
                b.count = 0;
                return r;
            };
            rc = g.each(list, [&](const Matrix& x, int64_t) -> int32_t {
                b.start[b.count++] = (uint32_t)at;
                at += ceil_div(x.rows * x.cols, kMomentumTile);
                b.start[b.count] = (uint32_t)at;
                return b.count < kMost ? (int32_t)ZS_OK : launch();
            });
            if (rc != ZS_OK) return rc;
            rc = launch();
            if (rc != ZS_OK) return rc;
        }
        {
            PackBatch b;
            std::memset(&b, 0, sizeof(b));
            b.sc = sc;
            b.sc_dev = sc_dev;
            b.norm_sq = norm_sq;
            b.ws = ws;
            b.inverse = most_partials > kPackPartials ? inverse : nullptr;
            b.partials = partials;
            int held = 0;
            auto launch = [&](PackBatch& x, int64_t tiles) {
                const hipError_t e = launch_pack(x, in_dtype == ZS_BF16, momentum, tiles, stream);
                if (x.inverse != nullptr) x.inverse += held;
                held = 0;
                return e;
            };
            int64_t partial = 0;
            Filler<PackBatch, decltype(launch)> fill(b, launch);
            rc = g.each(list, [&](const Matrix& x, int64_t unit) -> int32_t {
                int e = 0;
                const int32_t failed = fill.add(stage_tiles(x.m(), x.n()), e);
                if (failed != ZS_OK) return failed;
                ++held;
                b.e[e] = PackEntry{{ptr_lo(x.in), ptr_lo(x.momentum)}, ptr_hi(x.in) | ptr_hi(x.momentum) << 16,
                                   (uint32_t)unit, (uint32_t)x.m(), x.n_tall(), (uint32_t)partial};
                partial += ceil_div(x.rows * x.cols, kMomentumTile);
                return ZS_OK;
            });
            if (rc != ZS_OK) return rc;
            rc = fill.flush();
            if (rc != ZS_OK) return rc;
        }

        // the steps: S, b S + c S^2, then X (the last one's to its destination)
        NsBatch b;
        std::memset(&b, 0, sizeof(b));
        b.ws = ws;
        b.sc_dev = sc_dev;
        b.a = sc.a;
        b.b = sc.b;
        b.c = sc.c;
        TileCount square, wide;
        int64_t skinny = 0, others = 0;
        g.each(list, [&](const Matrix& x, int64_t) {
            if (x.m() <= kSkinny) {
                ++skinny;
                return ZS_OK;
            }
            ++others;
            square.add(pad_side(x.m()), pad_side(x.m()), x.m(), true);
            wide.add(pad_side(x.m()), pad_side(x.n()), x.m(), false);
            return ZS_OK;
        });
        constexpr int64_t kMost = sizeof(b.e) / sizeof(b.e[0]);
        const int square_size = square.size(kMost), wide_size = wide.size(kMost);
        // one launch of the steps over the matrices of one kind; tiles(matrix): its workgroups
        auto phase = [&](bool of_skinny, auto tiles, auto launch) -> int32_t {
            Filler<NsBatch, decltype(launch)> fill(b, launch);
            const int32_t r = g.each(list, [&](const Matrix& x, int64_t unit) -> int32_t {
                if ((x.m() <= kSkinny) != of_skinny) return ZS_OK;
                int e = 0;
                const int32_t failed = fill.add(tiles(x), e);
                if (failed != ZS_OK) return failed;
                b.e[e] = NsEntry{(uint32_t)unit, (uint32_t)x.m(), (uint32_t)x.n()};
                return ZS_OK;
            });
            return r != ZS_OK ? r : fill.flush();
        };
        for (int32_t step = 0; step < steps && others > 0; ++step) {
            b.which = step % 2;
            for (int kind_of = kNsGram; kind_of <= (step + 1 < steps ? kNsUpdate : kNsPoly); ++kind_of) {
                const int size = kind_of == kNsUpdate ? wide_size : square_size;
                rc = phase(false,
                           [&](const Matrix& x) {
                               TileCount one;
                               one.add(pad_side(x.m()), pad_side(x.n()), 0, kind_of != kNsUpdate);
                               return one.of[size];
                           },
                           [&](const NsBatch& x, int64_t tiles) { return launch_ns(x, kind_of, size, tiles, stream); });
                if (rc != ZS_OK) return rc;
            }
        }
        const int32_t at_once = sc_dev == nullptr ? skinny_steps_at_once(sc.a) : kSkinnySteps;
        for (int32_t done = 0; done < steps && skinny > 0; done += at_once) {
            b.which = done > 0;
            b.steps = std::min(steps - done, at_once);
            rc = phase(true, [&](const Matrix& x) { return SkinnyPlace(x.n()).chunks; },
                       [&](const NsBatch& x, int64_t tiles) { return launch_skinny_gram(x, tiles, stream); });
            if (rc != ZS_OK) return rc;
            rc = phase(true, [&](const Matrix&) { return (int64_t)1; },
                       [&](const NsBatch& x, int64_t tiles) { return launch_skinny_steps(x, tiles, stream); });
            if (rc != ZS_OK) return rc;
        }
        FinalBatch f;
        std::memset(&f, 0, sizeof(f));
        f.ws = ws;
        f.sc = sc;
        f.sc_dev = sc_dev;
        f.norm_sq = norm_sq;
        f.which = (steps - 1) % 2;
        for (int of_skinny = 0; of_skinny < 2; ++of_skinny) {
            const int size = of_skinny ? (int)kTile64 : wide_size;
            auto launch = [&](const FinalBatch& x, int64_t tiles) {
                return launch_ns_final(x, kind, size, of_skinny != 0, tiles, stream);
            };
            Filler<FinalBatch, decltype(launch)> fill(f, launch);
            rc = g.each(list, [&](const Matrix& x, int64_t unit) -> int32_t {
                if ((x.m() <= kSkinny) != (of_skinny != 0)) return ZS_OK;
                TileCount one;
                one.add(x.m(), x.n(), 0, false);
                int e = 0;
                const int32_t failed = fill.add(one.of[size], e);
                if (failed != ZS_OK) return failed;
                f.e[e] = FinalEntry{(uint32_t)unit, (uint32_t)x.m(), x.n_tall(), {ptr_lo(x.out), ptr_lo(x.copy)},
                                    ptr_hi(x.out) | ptr_hi(x.copy) << 16, x.scale};
                return ZS_OK;
            });
            if (rc != ZS_OK) return rc;
            rc = fill.flush();
            if (rc != ZS_OK) return rc;
        }
    }
    return ZS_OK;
}

int32_t check_muon(const zs_muon* hp) {
    if (hp == nullptr) return ZS_EINVAL;
    if (!(hp->lr >= 0.0) || !finite_float(hp->lr)) return ZS_EINVAL;
    if (!(hp->momentum >= 0.0 && (float)hp->momentum < 1.0f)) return ZS_EINVAL;
    if (!(hp->weight_decay >= 0.0) || !finite_float(hp->lr * hp->weight_decay)) return ZS_EINVAL;
    if (!coefficient_ok(hp->a) || !coefficient_ok(hp->b) || !coefficient_ok(hp->c) || !eps_ok(hp->eps)) return ZS_EINVAL;
    if (!positive_float(hp->grad_scale)) return ZS_EINVAL;
    if (std::isnan(hp->max_norm) || !(hp->extra_norm_sq >= 0.0)) return ZS_EINVAL;
    if (hp->nesterov != 0 && hp->nesterov != 1) return ZS_EINVAL;
    return hp->ns_steps >= 1 && hp->ns_steps <= ZS_NS_MAX_STEPS ? ZS_OK : ZS_EINVAL;
}

MuonScalars make_muon_scalars(const zs_muon* hp) {
    MuonScalars c;
    std::memset(&c, 0, sizeof(c));
    c.momentum = (float)hp->momentum;
    c.one_minus_momentum = (float)(1.0 - hp->momentum);
    c.decay = (float)(1.0 - hp->lr * hp->weight_decay);
    c.lr = (float)hp->lr;
    c.a = (float)hp->a;
    c.b = (float)hp->b;
    c.c = (float)hp->c;
    c.grad_scale = (float)hp->grad_scale;
    c.nesterov = hp->nesterov;
    c.clip = hp->max_norm > 0.0;
    c.eps = hp->eps;
    c.max_norm = hp->max_norm;
    c.extra_norm_sq = hp->extra_norm_sq;
    return c;
}

int32_t muon_step(const zs_muon* hp, const zs_muon_scalars* sc_dev, int32_t steps, const zs_muon_matrix* list,
                  int32_t count, int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev, void* workspace,
                  int64_t workspace_bytes, void* hip_stream) {
    const int64_t need = ns_workspace(list, count);
    if (need < 0 || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return ZS_EINVAL;
    if (steps < 1 || steps > ZS_NS_MAX_STEPS) return ZS_EINVAL;
    if (norm_sq_dev != nullptr && !aligned(norm_sq_dev, 8)) return ZS_EINVAL;
    if (sc_dev != nullptr && !aligned(sc_dev, 8)) return ZS_EINVAL;
    const int32_t rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != ZS_OK) return rc;
    Ranges ranges;
    if (!ranges.reserve(count, 5)) return ZS_EINVAL;
    for (int32_t k = 0; k < count; ++k) {
        const zs_muon_matrix& x = list[k];
        const int64_t n = x.rows * x.cols;
        if (n == 0) continue;
        if (!typed(x.param, param_dtype) || !typed(x.grad, grad_dtype) || !typed(x.momentum, ZS_F32)) return ZS_EINVAL;
        if (x.param_bf16 != nullptr && (param_dtype == ZS_BF16 || !typed(x.param_bf16, ZS_BF16))) return ZS_EINVAL;
        if (!finite_float(x.scale)) return ZS_EINVAL;
        ranges.add(0, x.param, n * elem_size(param_dtype), true);
        ranges.add(1, x.grad, n * elem_size(grad_dtype), false);
        ranges.add(2, x.momentum, n * 4, true);
        ranges.add(3, x.param_bf16, n * 2, true);
    }
    if (count > 0) ranges.add(4, workspace, need, true);
    ranges.add_read(norm_sq_dev, 8);
    ranges.add_read(sc_dev, (int64_t)sizeof(zs_muon_scalars));
    if (ranges.clash()) return ZS_EOVERLAP;
    MuonScalars sc;
    std::memset(&sc, 0, sizeof(sc));
    if (sc_dev == nullptr) sc = make_muon_scalars(hp);
    return run_ns(list, count, grad_dtype, param_dtype == ZS_BF16 ? kFinalParamBf16 : kFinalParamF32, steps, sc,
                  reinterpret_cast<const MuonScalars*>(sc_dev), norm_sq_dev, static_cast<char*>(workspace), hip_stream);
}

}  // namespace

extern "C" {

int64_t product_add_matrices_workspace_bytes(const zs_product* list, int32_t count, int32_t in_dtype, int32_t flags) {
    if ((flags & ~(ZS_TRANSPOSE_A | ZS_TRANSPOSE_B)) != 0) return -1;
    return products_workspace(list, count, in_dtype, flags);
}

int32_t product_add_matrices(const zs_product* list, int32_t count, int32_t in_dtype, int32_t c_dtype, int32_t d_dtype,
                             int32_t flags, double alpha, double beta, void* workspace, int64_t workspace_bytes,
                             void* hip_stream) {
    if ((flags & ~(ZS_TRANSPOSE_A | ZS_TRANSPOSE_B)) != 0) return ZS_EINVAL;
    return products(list, count, in_dtype, c_dtype, d_dtype, flags, alpha, beta, workspace, workspace_bytes, hip_stream);
}

int64_t gram_add_matrices_workspace_bytes(const zs_gram* list, int32_t count, int32_t in_dtype) {
    return products_workspace(list, count, in_dtype, 0);
}

int32_t gram_add_matrices(const zs_gram* list, int32_t count, int32_t in_dtype, int32_t d_dtype, double alpha, double beta,
                          void* workspace, int64_t workspace_bytes, void* hip_stream) {
    return products(list, count, in_dtype, d_dtype, d_dtype, 0, alpha, beta, workspace, workspace_bytes, hip_stream);
}

int64_t orthogonalize_matrices_workspace_bytes(const zs_orthogonal* list, int32_t count) { return ns_workspace(list, count); }

int32_t orthogonalize_matrices(const zs_orthogonal* list, int32_t count, int32_t in_dtype, int32_t steps, double a, double b,
                               double c, double eps, void* workspace, int64_t workspace_bytes, void* hip_stream) {
    const int64_t need = ns_workspace(list, count);
    if (need < 0 || !dtype_ok(in_dtype) || steps < 1 || steps > ZS_NS_MAX_STEPS) return ZS_EINVAL;
    if (!coefficient_ok(a) || !coefficient_ok(b) || !coefficient_ok(c) || !eps_ok(eps)) return ZS_EINVAL;
    const int32_t rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != ZS_OK) return rc;
    Ranges ranges;
    if (!ranges.reserve(count, 3)) return ZS_EINVAL;
    for (int32_t k = 0; k < count; ++k) {
        const int64_t n = list[k].rows * list[k].cols;
        if (n == 0) continue;
        if (!typed(list[k].in, in_dtype) || !typed(list[k].out, ZS_BF16)) return ZS_EINVAL;
        ranges.add(0, list[k].in, n * elem_size(in_dtype), false);
        ranges.add(1, list[k].out, n * 2, true);
    }
    if (count > 0) ranges.add(2, workspace, need, true);
    if (ranges.clash()) return ZS_EOVERLAP;
    MuonScalars sc;
    std::memset(&sc, 0, sizeof(sc));
    sc.a = (float)a;
    sc.b = (float)b;
    sc.c = (float)c;
    sc.eps = eps;
    return run_ns(list, count, in_dtype, kFinalBf16, steps, sc, nullptr, nullptr, static_cast<char*>(workspace), hip_stream);
}

int64_t muon_step_matrices_workspace_bytes(const zs_muon_matrix* list, int32_t count) { return ns_workspace(list, count); }

int32_t muon_scalars(const zs_muon* hp, zs_muon_scalars* out) {
    const int32_t rc = check_muon(hp);
    if (rc != ZS_OK || out == nullptr) return ZS_EINVAL;
    const MuonScalars c = make_muon_scalars(hp);
    std::memcpy(out, &c, sizeof(c));
    return ZS_OK;
}

int32_t muon_step_matrices(const zs_muon* hp, const zs_muon_matrix* list, int32_t count, int32_t param_dtype,
                           int32_t grad_dtype, const double* norm_sq_dev, void* workspace, int64_t workspace_bytes,
                           void* hip_stream) {
    if (check_muon(hp) != ZS_OK) return ZS_EINVAL;
    return muon_step(hp, nullptr, hp->ns_steps, list, count, param_dtype, grad_dtype, norm_sq_dev, workspace,
                     workspace_bytes, hip_stream);
}

int32_t muon_step_matrices_dev(const zs_muon_scalars* scalars_dev, int32_t ns_steps, const zs_muon_matrix* list,
                               int32_t count, int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev,
                               void* workspace, int64_t workspace_bytes, void* hip_stream) {
    if (scalars_dev == nullptr) return ZS_EINVAL;
    return muon_step(nullptr, scalars_dev, ns_steps, list, count, param_dtype, grad_dtype, norm_sq_dev, workspace,
                     workspace_bytes, hip_stream);
}

}  // extern "C"
