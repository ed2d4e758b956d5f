// Calls over lists of matrices: the tables that travel in the kernel arguments
// and the layout of the workspace (internal).
#pragma once

#include "tensors.h"

namespace zs {

// Matrices in the workspace have both sides padded to whole k tiles with zeros,
// so the products need no tails.  Those of the Newton-Schulz steps lie in blocks of
// 64 x 64 (mfma_tile.h): what a tile reads and writes is a few pieces of 8 KiB
// instead of hundreds of rows some pages apart.
constexpr int64_t kPadSide = 64;
__host__ __device__ __forceinline__ int64_t pad_side(int64_t n) { return (n + kPadSide - 1) / kPadSide * kPadSide; }

// Tiles of a product, from large to small (products.hip).
enum TileSize : int { kTile256 = 0, kTile128 = 1, kTile64 = 2 };
inline int64_t tile_side(int size) { return 256 >> size; }

// --- products over the caller's matrices ------------------------------------
// a and b are in the form that the kernels take: k a multiple of 64 (zeros past
// the caller's k), 16-byte aligned rows.
struct ProductEntry {
    uint32_t lo[4];        // a, b, c, d
    uint32_t hi[2];        // a | b << 16, c | d << 16
    uint32_t m, n;
    uint32_t k_tiles;
    uint32_t lda, ldb;     // elements
};
struct ProductBatch {
    ListTable<80> tab;
    ProductEntry e[80];
    float alpha, beta;
    int32_t c_bf16, d_bf16;
};
static_assert(sizeof(ProductBatch) <= 4096, "kernel arguments");
// b_cols: b is k x n (else n x k).  sym: b is a's equal in value, m == n, and
// tiles above the diagonal mirror those below.  split: k is three products of split
// values.
hipError_t launch_products(const ProductBatch& b, int size, bool b_cols, bool sym, bool split, int64_t tiles,
                           hipStream_t stream);

// Copies of operands into the kernels' form.
enum StageKind : int { kStagePlain = 0, kStageHiHiLo = 1, kStageHiLoHi = 2 };
struct StageEntry {
    uint32_t lo[2];        // source, destination
    uint32_t hi;           // source | destination << 16
    uint32_t rows, cols;   // of the destination, without padding
};
struct StageBatch {
    ListTable<150> tab;
    StageEntry e[150];
};
static_assert(sizeof(StageBatch) <= 4096, "kernel arguments");
// destination: rows x cols padded on both sides, three times so along k for the
// split kinds (k is the rows for k_rows, else the columns).  transposed: the
// source is cols x rows.
hipError_t launch_stage(const StageBatch& b, int src_bf16, int kind, bool k_rows, bool transposed, int64_t tiles,
                        hipStream_t stream);
inline int64_t stage_tiles(int64_t rows, int64_t cols) { return pad_side(rows) / kPadSide * (pad_side(cols) / kPadSide); }

// --- Newton-Schulz steps ------------------------------------------------------
// X lies short side x long side, whatever way the caller's matrix lies.  One
// matrix's place in the workspace, from its base: X's two halves (first and
// second fp16 of each pair), twice (a step reads one and writes the other),
// then S and b S + c S^2.
constexpr int64_t kNsUnit = 8192;     // every part is a multiple of it
constexpr float kNsScale = 256.0f;    // of what is held in fp16
// A pair's second value is the remainder times this: as large as the first one, so
// that both stay normal numbers where X's values are small (a 4096 x 11008 matrix of
// norm 1 has values of 2^-13).
constexpr float kNsLow = 2048.0f;
// The value is held in a register of its own first: left to itself the compiler
// rounds the first half from the unrounded product and takes the remainder against
// a second conversion, which differ near ties.
__device__ __forceinline__ void split_f16(float x, _Float16& hi, _Float16& lo) {
    asm("" : "+v"(x));
    hi = (_Float16)x;
    lo = (_Float16)__builtin_fmaf((float)hi, -kNsLow, x * kNsLow);
}
struct NsEntry {
    uint32_t base;         // in kNsUnit
    uint32_t m, n;         // short, long side
};
struct NsPlace {
    int64_t mp, np, x;     // padded sides, bytes of one half of X
    __host__ __device__ __forceinline__ NsPlace(int64_t m, int64_t n) : mp(pad_side(m)), np(pad_side(n)), x(mp * np * 2) {}
    __host__ __device__ __forceinline__ int64_t hi(int which) const { return which * 2 * x; }
    __host__ __device__ __forceinline__ int64_t lo(int which) const { return which * 2 * x + x; }
    __host__ __device__ __forceinline__ int64_t s() const { return 4 * x; }
    __host__ __device__ __forceinline__ int64_t poly() const { return 4 * x + mp * mp * 2; }
    __host__ __device__ __forceinline__ int64_t bytes() const { return 4 * x + 2 * mp * mp * 2; }
};
// A matrix whose short side is one k tile or less goes another way: its steps
// are polynomials of S = X X^T, a 64 x 64 matrix, so one workgroup forms their
// product Q in fp32 from the pairs' S, and Q X is the result.  X is read twice
// instead of ten times, in 5 launches instead of 17, and nothing is rounded to
// fp16 alone: with few singular values the roundings of the other way do not
// average out (up to 9e-3 of a 2 x 3 matrix; this way 1e-5).
// That holds for a few steps at a time.  S is off by 2^-23 of its largest value, and
// its small and null values, that error with them, grow by a^2 a step, below zero too,
// where the polynomial has no bound (3.4445: a 64 x 256 matrix of rank 8 off by 1e-4 after
// 5 steps, 0.4 after 8, NaN after 12).  And Q, a pair, is off by 2^-22 of its own largest
// value, a^steps there.  So X becomes Q X, and S is formed anew from it, before |a|^steps
// passes kSkinnyGrowth, and after kSkinnySteps steps: Q is off by 512 * 2^-22 = 1.2e-4 at
// most then, and S, where X is small, by 512^2 / a^2 * 2^-23 = 3e-3.  Every workgroup of the
// next sum of S does so for its columns.  Where a is in device memory the launches cannot
// go by it (a captured step's coefficients may change) and are those of kSkinnySteps;
// within them, for |a| above 3.48, the workgroup that forms Q does so for all columns,
// which takes longer (5 steps with a = 4.08 of 64 x 11008: 114 us, so 564).
constexpr int64_t kSkinny = kPadSide;
constexpr int32_t kSkinnySteps = 5;
constexpr float kSkinnyGrowth = 512.0f;
__host__ __device__ __forceinline__ int32_t skinny_steps_at_once(float a) {
    const float slope = a < 0.0f ? -a : a;
    int32_t steps = 1;
    for (float grown = slope * slope; steps < kSkinnySteps && grown <= kSkinnyGrowth; grown *= slope) ++steps;
    return steps;
}
// Its place: X's first values, second values and first values again (together the
// 192 x np right operand of Q X), the partial sums of S, Q as its left operand
// (64 x 192), Q's scale.
struct SkinnyPlace {
    int64_t np, x, chunk, chunks;   // chunk: k tiles of one partial sum
    __host__ __device__ __forceinline__ explicit SkinnyPlace(int64_t n) : np(pad_side(n)), x(kSkinny * np * 2) {
        const int64_t tiles = np / kPadSide;
        chunk = tiles > 16 * 128 ? (tiles + 127) / 128 : 16;
        chunks = (tiles + chunk - 1) / chunk;
    }
    static constexpr int64_t kPart = kSkinny * kSkinny * 4;
    __host__ __device__ __forceinline__ int64_t parts() const { return 3 * x; }
    __host__ __device__ __forceinline__ int64_t q() const { return 3 * x + chunks * kPart; }
    __host__ __device__ __forceinline__ int64_t scale() const { return q() + 3 * kSkinny * kSkinny * 2; }
    __host__ __device__ __forceinline__ int64_t bytes() const { return scale() + kNsUnit; }
};
inline int64_t ns_bytes(int64_t m, int64_t n) { return m <= kSkinny ? SkinnyPlace(n).bytes() : NsPlace(m, n).bytes(); }

struct MuonScalars {       // zs_muon_scalars
    float momentum, one_minus_momentum, decay, lr;
    float a, b, c;
    float grad_scale;
    int32_t nesterov, clip;
    double eps;
    double max_norm, extra_norm_sq;
};
struct NsBatch {
    ListTable<240> tab;
    NsEntry e[240];
    char* ws;
    const MuonScalars* sc_dev;
    float a, b, c;         // unless sc_dev is set
    int32_t which;         // the X that is read; skinny matrices: 1 where X is to become Q X first
    int32_t steps;         // skinny matrices: up to the next sum of S
};
static_assert(sizeof(NsBatch) <= 4096, "kernel arguments");
enum NsPhase : int { kNsGram = 0, kNsPoly = 1, kNsUpdate = 2 };
hipError_t launch_ns(const NsBatch& b, int phase, int size, int64_t tiles, hipStream_t stream);
// a workgroup per partial sum of S (after X <- Q X where b.which is 1); a workgroup per matrix
hipError_t launch_skinny_gram(const NsBatch& b, int64_t tiles, hipStream_t stream);
hipError_t launch_skinny_steps(const NsBatch& b, int64_t count, hipStream_t stream);

// The last step: X goes to its destination instead.
constexpr uint32_t kTall = 0x80000000u;
struct FinalEntry {
    uint32_t base, m, n;   // n: kTall set where the caller's matrix is long side x short side
    uint32_t lo[2];        // param (or output), re-cast
    uint32_t hi;           // param | re-cast << 16
    float scale;
};
struct FinalBatch {
    ListTable<118> tab;
    FinalEntry e[118];
    char* ws;
    const MuonScalars* sc_dev;
    const double* norm_sq;
    MuonScalars sc;        // unless sc_dev is set
    int32_t which;
};
static_assert(sizeof(FinalBatch) <= 4096, "kernel arguments");
enum FinalKind : int { kFinalBf16 = 0, kFinalParamF32 = 1, kFinalParamBf16 = 2 };   // the output alone; a parameter's step
hipError_t launch_ns_final(const FinalBatch& b, int kind, int size, bool skinny, int64_t tiles, hipStream_t stream);

// --- what comes before them ---------------------------------------------------
// New momentum, and the squares of u per tile of kMomentumTile elements (binary64).
constexpr int64_t kMomentumTile = 4096;
struct MomentumEntry {
    uint32_t lo[2];        // gradient (or input), momentum
    uint32_t hi;           // gradient | momentum << 16
    uint32_t numel;
};
struct MomentumBatch {
    ListTable<180> tab;
    MomentumEntry e[180];
    double* partials;      // of the launch's first tile
    const MuonScalars* sc_dev;
    const double* norm_sq;
    MuonScalars sc;
};
static_assert(sizeof(MomentumBatch) <= 4096, "kernel arguments");
hipError_t launch_momentum(const MomentumBatch& b, int grad_bf16, bool momentum, int64_t tiles, hipStream_t stream);

// kNsScale / max(norm, eps) of each matrix from its partials
struct NormsBatch {
    uint32_t start[960 + 1];   // first partial of each matrix, and the last one's end
    uint32_t count;
    const double* partials;
    float* inverse;
    const MuonScalars* sc_dev;
    double eps;                // unless sc_dev is set
};
static_assert(sizeof(NormsBatch) <= 4096, "kernel arguments");
hipError_t launch_inverse_norms(const NormsBatch& b, hipStream_t stream);

// u, scaled, into X's halves
struct PackEntry {
    uint32_t lo[2];        // gradient (or input), momentum
    uint32_t hi;
    uint32_t base, m, n;   // n: kTall as in FinalEntry
    uint32_t partial;      // the matrix's first one
};
// Where no matrix of a group has more partials than this, the norm is formed where it is
// used (in every workgroup anew, in the same order): a launch less, one matrix of
// 1024 x 1024 39.5 -> 37.3 us for one step, lists of 64 and 400 of them as before.  More
// partials would be more than one load a thread, in each of a matrix's workgroups.
constexpr int64_t kPackPartials = kBlock;
struct PackBatch {
    ListTable<118> tab;
    PackEntry e[118];
    char* ws;
    const float* inverse;  // of the first entry; NULL: from the partials
    const double* partials;
    const MuonScalars* sc_dev;
    const double* norm_sq;
    MuonScalars sc;
};
static_assert(sizeof(PackBatch) <= 4096, "kernel arguments");
hipError_t launch_pack(const PackBatch& b, int grad_bf16, bool momentum, int64_t tiles, hipStream_t stream);

}  // namespace zs
