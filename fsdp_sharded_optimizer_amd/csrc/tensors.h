// Calls over lists of tensors: the tables that travel in the kernel arguments
// and how a workgroup finds its tensor (internal).
#pragma once

#include "zs_common.h"

namespace zs {

// One launch covers up to N tensors.  A tensor's elements are cut in tiles;
// workgroups are laid out tensor after tensor, and start[t] is the first
// workgroup of tensor t (of the launch's end for the one past the last, then
// kNoTile).  A workgroup finds its tensor in three dependent rounds of scalar
// loads: the tensor that a 32nd of the launch begins in, the next 8 starts
// (again only where 8 small tensors begin in one such part before the
// workgroup's), and the tensor's record. Against a scan of every eighth start
// and then of 8, as the compiler wrote them (through vector registers): the norm
// of 855M gradients 266 -> 250 us.
constexpr int kListBuckets = 32;
constexpr int kListScan = 8;
constexpr uint32_t kNoTile = 0xFFFFFFFFu;
template <int N>
struct ListTable {
    static constexpr int kMax = N;
    static constexpr int kBits = N <= 256 ? 8 : 16, kPerWord = 32 / kBits;
    uint32_t shift;                             // workgroup w is in part w >> shift
    uint32_t bucket[kListBuckets / kPerWord];   // the tensor of each part's first workgroup
    uint32_t start[N + kListScan];
};

// t + (w >= start) in two scalar instructions (the compiler takes the carry
// through vector registers, about five times as long).  The look-up and the order of
// tiles are host functions too, for checks of the tables without a GPU.
__device__ __forceinline__ void count_past(uint32_t& t, uint32_t w, uint32_t start) {
    asm("s_cmp_ge_u32 %1, %2\n\ts_addc_u32 %0, %0, 0" : "+s"(t) : "s"(w), "s"(start) : "scc");
}
__host__ inline void count_past(uint32_t& t, uint32_t w, uint32_t start) { t += w >= start; }

template <int N>
__host__ __device__ __forceinline__ uint32_t find_tensor(const ListTable<N>& tab, uint32_t w, uint32_t& first) {
    const uint32_t part = w >> tab.shift;
    constexpr uint32_t kPer = ListTable<N>::kPerWord, kBits = ListTable<N>::kBits;
    uint32_t t = tab.bucket[part / kPer] >> (kBits * (part % kPer)) & ((1u << kBits) - 1u), from;
    do {
        from = t;
        const uint32_t* const next = tab.start + from + 1;   // one load of all 8
        uint32_t s[kListScan];
#pragma unroll
        for (int k = 0; k < kListScan; ++k) s[k] = next[k];
#pragma unroll
        for (int k = 0; k < kListScan; ++k) count_past(t, w, s[k]);
    } while (t == from + kListScan);
    first = tab.start[t];
    return t;
}

// The tile of workgroup w of n when an XCD takes runs of 4 consecutive tiles
// (gfx950 deals workgroups to its 8 XCDs in turn).  Where written streams do not
// start on cache lines, neighbouring tiles write parts of one line, which is
// then put together in one XCD's L2 instead of in memory: 405M moments read out
// to odd offsets 507 -> 433 us, the 8-bit step 80 -> 76 at 25M fp32 parameters
// (the same at 405M, whose parameters' lines are kept as well).  On aligned
// tensors it costs 2-7 %.
__host__ __device__ __forceinline__ uint32_t tile_in_runs(uint32_t w, uint32_t n) {
    constexpr uint32_t kRun = 4, kAll = 8 * kRun;
    const uint32_t base = w / kAll * kAll, i = w % kAll;
    return base + kAll > n ? w : base + (i % 8) * kRun + i / 8;
}

// A device address in 48 bits: its low word, and its upper 16 bits as one half
// of a word.  A record of five pointers and a length is then 36 bytes, and the 4
// KiB of kernel arguments hold 98 of them (with whole pointers 64).
template <typename T>
__device__ __forceinline__ T* unpack_ptr(uint32_t lo, uint32_t hi16) {
    // global memory, said so: accesses through a pointer made from an integer
    // are flat ones otherwise, which also wait for LDS
    typedef __attribute__((address_space(1))) T Global;
    return (T*)(Global*)((uint64_t)(hi16 & 0xFFFFu) << 32 | lo);
}
inline bool packable(const void* p) { return (reinterpret_cast<uintptr_t>(p) >> 48) == 0; }
inline uint32_t ptr_lo(const void* p) { return (uint32_t)reinterpret_cast<uintptr_t>(p); }
inline uint32_t ptr_hi(const void* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) >> 32); }

// --- accesses at any element alignment -------------------------------------
// gfx950 serves vector accesses at any byte address; the types tell the
// compiler the weaker alignment, so tensors at odd offsets take the same
// 128- and 64-bit instructions as aligned ones.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_to_f32(x); }
template <bool BF16> struct GradType { using T = float; };
template <> struct GradType<true> { using T = uint16_t; };

// Four consecutive elements of an fp32 or bf16 stream, as fp32.  KEEP: read so
// that the caches keep the lines, instead of as a stream (a template argument:
// of two branches that differ in this alone the compiler makes one load).
template <bool KEEP = false>
__device__ __forceinline__ f32x4 ld4(const float* p) {
    const f32x4_any* const q = reinterpret_cast<const f32x4_any*>(p);
    if constexpr (KEEP) return *q;
    else return __builtin_nontemporal_load(q);
}
template <bool KEEP>
__device__ __forceinline__ u32x2 ld_u32x2_any(const void* p) {
    const u32x2_any* const q = static_cast<const u32x2_any*>(p);
    if constexpr (KEEP) return *q;
    else return __builtin_nontemporal_load(q);
}
template <bool KEEP>
__device__ __forceinline__ u32x4 ld_u32x4_any(const void* p) {
    const u32x4_any* const q = static_cast<const u32x4_any*>(p);
    if constexpr (KEEP) return *q;
    else return __builtin_nontemporal_load(q);
}
template <bool KEEP = false>
__device__ __forceinline__ f32x4 ld4(const uint16_t* p) {
    const u32x2 w = ld_u32x2_any<KEEP>(p);
    return f32x4{bf16_to_f32(w.x & 0xFFFFu), bf16_to_f32(w.x >> 16), bf16_to_f32(w.y & 0xFFFFu),
                 bf16_to_f32(w.y >> 16)};
}
__device__ __forceinline__ void st4(float* p, const f32x4& x) {
    __builtin_nontemporal_store(f32x4_any(x), reinterpret_cast<f32x4_any*>(p));
}
__device__ __forceinline__ void st4(uint16_t* p, const f32x4& x) {
    const u32x2 w = {pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w)};
    __builtin_nontemporal_store(u32x2_any(w), reinterpret_cast<u32x2_any*>(p));
}
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(uint16_t* p, float x) { *p = (uint16_t)f32_to_bf16_rne(x); }

// A workgroup count keeps a launch below 2^32 work-items at up to 256 threads.
constexpr int64_t kListMaxTiles = (int64_t(1) << 32) / 256 - 1;   // so starts fit 31 bits as well

// A tensor of more than kLaunchElems elements is cut into entries of that many
// (a multiple of every tile), so an entry's numel fits 32 bits.

// Whether a list's gradients are read so that the last-level cache (256 MiB)
// keeps them: they fit it, the norm reads them before the step does, and a
// backward pass wrote the last of them shortly before that.  The other streams go
// past it.  Norm and step of bf16 gradients as streams / kept, us: 34M parameters
// 132 / 124, 76M 279 / 261, 124M 454 / 423 (fp32 ones with re-casts 164 / 159, 354 /
// 338, 564 / 543; 8-bit moments 153 / 148 at 76M), 148M the same, 190M 690 / 696.
constexpr int64_t kKeepBytes = int64_t(240) << 20;
inline bool keep_grads(int64_t grad_bytes) { return grad_bytes <= kKeepBytes; }

// --- the squared norm -----------------------------------------------------
// A tensor's tiles are whole but the last one, so its record holds the elements
// of that one alone (less 1): 8 bytes, and the 291 tensors of a 7B model are one
// launch (25M bf16 gradients in 290 tensors: 21.9 -> 14.1 us, with one launch less for
// the sum of the partials as well).
struct NormEntry {
    uint32_t lo, hi_tail;   // tail << 16
};
struct NormBatch {
    ListTable<328> tab;
    NormEntry e[328];
};
static_assert(sizeof(NormBatch) <= 4072, "kernel arguments");
int64_t norm_tile_elems(int grad_bf16);   // elements per workgroup (one binary64 partial each)
hipError_t launch_norm_tensors(const NormBatch& b, int grad_bf16, bool keep, int64_t tiles, float scale,
                               double* partials, hipStream_t stream);
// Up to this many partials one workgroup adds in one launch; beyond it the two of
// launch_sum_partials, with its stage.
constexpr int64_t kListSumOneGroup = 16384;
hipError_t launch_list_sum(const double* partials, int64_t count, double* stage, double* out, hipStream_t stream);

// --- AdamW, fp32 moments --------------------------------------------------
// Tile 0 of a tensor starts `shift` elements before its first one, for the
// alignment of the tiles (less than one tile).
struct AdamwEntry {
    uint32_t lo[5];   // param, grad, exp_avg, exp_avg_sq, bf16 re-cast (0: none)
    uint32_t hi[3];   // param | grad << 16, exp_avg | exp_avg_sq << 16, re-cast | shift << 16
    uint32_t numel;
};
struct AdamwBatch {
    ListTable<98> tab;
    AdamwEntry e[98];
    const AdamwScalars* sc_dev;
    const double* norm_sq;       // nullable
    AdamwScalars sc;             // unless sc_dev is set
};
constexpr int64_t kListTile = 256;
static_assert(sizeof(AdamwBatch) <= 4096, "kernel arguments");
// keep: of the gradients; off_line: most tiles start off a cache line in some stream
hipError_t launch_adamw_tensors(const AdamwBatch& b, int param_bf16, int grad_bf16, bool keep, bool off_line,
                                int64_t tiles, hipStream_t stream);

// --- 8-bit moments --------------------------------------------------------
// Layout of one tensor's buffer of n elements, P = n rounded up to kQ8Pad:
// 2 P bytes of codes (their order is in q8.h), then two bytes per block (exp_avg's
// e, exp_avg_sq's e).
constexpr int64_t kQ8Block = 256;
constexpr int64_t kQ8Pad = 512;
__host__ __device__ __forceinline__ int64_t q8_padded(int64_t n) { return (n + kQ8Pad - 1) / kQ8Pad * kQ8Pad; }

struct Q8Scalars {   // zs_adamw_q8_scalars
    AdamwScalars adamw;
    uint32_t key;
    uint32_t reserved;
};

// A record is 26 bytes with its tile start, so that the 291 tensors of a 7B
// model are two launches (with whole pointers and lengths 98 to a launch, three:
// 25M parameters in 290 tensors, step and read-out 78 -> 72 and 39 -> 35 us;
// lists of a few long tensors 0-1 % slower).  Of an address the low word and
// bits 32-39; bits 40-47 are the launch's (one window of 1 TiB for each stream;
// another one starts another launch).  A tensor's tiles are whole but the last,
// whose elements (less 1) are the tail.  Records are of consecutive tensors of
// the caller's list, those without elements included (no tiles).  A piece of a
// tensor longer than kLaunchElems is alone in its launch.
struct Q8Entry {
    uint32_t lo[4];       // step: param, grad, state, bf16 re-cast; conversions: exp_avg, exp_avg_sq, state
    uint32_t hi;          // a byte of each
};
constexpr uint32_t kQ8Tail = 0x1FF, kQ8Has0 = 0x8000, kQ8Has1 = 0x4000, kQ8Has3 = 0x2000;   // which pointers are not NULL
struct Q8Batch {
    ListTable<150> tab;
    Q8Entry e[150];
    uint32_t tail[75];           // 16 bits each: the tail and kQ8Has bits
    uint32_t runs;               // not 0: workgroups take their tiles in runs (tile_in_runs)
    uint32_t top;                // bits 40-47 of the addresses, a byte of each
    uint32_t index;              // the first record's place in the caller's list
    uint32_t off, padded;        // a piece: elements before it in units of kLaunchElems, the whole tensor's padded
                                 // length in units of kQ8Pad; otherwise 0
    const Q8Scalars* sc_dev;
    const double* norm_sq;       // nullable
    Q8Scalars sc;                // the conversions use the key alone
};
static_assert(sizeof(Q8Batch) <= 4096, "kernel arguments");
hipError_t launch_adamw_q8(const Q8Batch& b, int param_bf16, int grad_bf16, bool keep, int64_t tiles,
                           hipStream_t stream);
hipError_t launch_q8_encode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream);
hipError_t launch_q8_decode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream);

}  // namespace zs
