// Calls over lists of tensors: the tables that travel in the kernel arguments
// and how a workgroup finds its tensor (internal).
#pragma once

#include "zs_common.h"

namespace zs {

// One launch covers up to kListMax tensors.  A tensor's elements are cut in
// tiles; workgroups are laid out tensor after tensor, and tile_start[t] is the
// first workgroup of tensor t (every entry past the last is UINT32_MAX).
// coarse[g] repeats tile_start[8g], so a workgroup finds its tensor with two
// rounds of scalar loads (8 coarse entries, then 8 fine ones) and then reads
// its record: three dependent scalar loads, against six or seven for a
// bisection, and a fourth of the comparisons of a scan over all 64.
constexpr int kListMax = 64;
constexpr int kListGroup = 8;
struct ListTable {
    uint32_t coarse[kListMax / kListGroup];
    uint32_t tile_start[kListMax];
};

__device__ __forceinline__ int find_tensor(const ListTable& tab, uint32_t w, uint32_t& first) {
    int g = 0;
#pragma unroll
    for (int k = 1; k < kListMax / kListGroup; ++k) g += w >= tab.coarse[k] ? 1 : 0;
    const int at = g * kListGroup;
    int t = at;
    first = tab.tile_start[at];
#pragma unroll
    for (int k = 1; k < kListGroup; ++k) {
        const uint32_t s = tab.tile_start[at + k];
        const bool past = w >= s;
        t += past ? 1 : 0;
        first = past ? s : first;
    }
    return t;
}

// --- accesses at any element alignment -------------------------------------
// gfx950 serves vector accesses at any byte address; the types tell the
// compiler the weaker alignment, so tensors at odd offsets take the same
// 128- and 64-bit instructions as aligned ones.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ u32x4 ld_stream_u32x4_any(const void* p) {
    return __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ u32x2 ld_stream_u32x2_any(const void* p) {
    return __builtin_nontemporal_load(static_cast<const u32x2_any*>(p));
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_to_f32(x); }
template <bool BF16> struct GradType { using T = float; };
template <> struct GradType<true> { using T = uint16_t; };

// Four consecutive elements of an fp32 or bf16 stream, as fp32.
__device__ __forceinline__ f32x4 ld4(const float* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(p));
}
__device__ __forceinline__ f32x4 ld4(const uint16_t* p) {
    const u32x2 w = ld_stream_u32x2_any(p);
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
constexpr int64_t kListMaxTiles = (int64_t(1) << 32) / 256 - 1;

// A tensor of more than kLaunchElems elements is cut into entries of that many
// (a multiple of every tile), so an entry's numel fits 32 bits.

// --- the squared norm -----------------------------------------------------
struct NormEntry {
    const void* grad;
    int64_t numel;
};
struct NormBatch {
    ListTable tab;
    NormEntry e[kListMax];
};
int64_t norm_tile_elems(int grad_bf16);   // elements per workgroup (one binary64 partial each)
hipError_t launch_norm_tensors(const NormBatch& b, int grad_bf16, int64_t tiles, float scale, double* partials,
                               hipStream_t stream);

// --- AdamW, fp32 moments --------------------------------------------------
// Tile 0 of a tensor starts `shift` elements before its first one, so that the
// other tiles start on cache lines of every stream that is read and written
// (0 where the tensor's streams do, or cannot all).
struct AdamwEntry {
    void* param;
    const void* grad;
    float* exp_avg;
    float* exp_avg_sq;
    uint16_t* copy;     // bf16 re-cast of an fp32 param, nullable
    uint32_t numel;
    uint32_t shift;
};
struct AdamwBatch {
    ListTable tab;
    AdamwScalars sc;             // unless sc_dev is set
    const AdamwScalars* sc_dev;
    const double* norm_sq;       // nullable
    AdamwEntry e[kListMax];
};
constexpr int64_t kListTile = 256;
static_assert(sizeof(AdamwBatch) <= 4096, "kernel arguments");
hipError_t launch_adamw_tensors(const AdamwBatch& b, int param_bf16, int grad_bf16, int64_t tiles,
                                hipStream_t stream);

// --- 8-bit moments --------------------------------------------------------
// Layout of one tensor's buffer of n elements, P = n rounded up to kQ8Pad:
// 2 P bytes of codes (their order is in q8.h), then two bytes per block (exp_avg's
// e, exp_avg_sq's e).  A workgroup takes kQ8Pad elements.
constexpr int64_t kQ8Block = 256;
constexpr int64_t kQ8Pad = 1024;
__host__ __device__ __forceinline__ int64_t q8_padded(int64_t n) { return (n + kQ8Pad - 1) / kQ8Pad * kQ8Pad; }

struct Q8Scalars {   // zs_adamw_q8_scalars
    AdamwScalars adamw;
    uint32_t key;
    uint32_t reserved;
};

// `off` elements of the tensor come before the entry's first, `padded` is the
// whole tensor's padded length (both in units of kQ8Pad); `state` is the whole
// tensor's buffer, the other pointers the entry's.  `index` is the tensor's
// place in the caller's list.
struct Q8Entry {
    void* param;        // encode: exp_avg source; decode: exp_avg destination (nullable)
    const void* grad;   // encode: exp_avg_sq source
    uint8_t* state;
    void* copy;         // the step's bf16 re-cast; decode: exp_avg_sq destination (nullable)
    uint32_t numel;
    uint32_t off;
    uint32_t padded;
    uint32_t index;
};
struct Q8Batch {
    ListTable tab;
    Q8Scalars sc;                // the conversions use the key alone
    const Q8Scalars* sc_dev;
    const double* norm_sq;       // nullable
    Q8Entry e[kListMax];
};
static_assert(sizeof(Q8Batch) <= 4096, "kernel arguments");
hipError_t launch_adamw_q8(const Q8Batch& b, int param_bf16, int grad_bf16, int64_t tiles, hipStream_t stream);
hipError_t launch_q8_encode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream);
hipError_t launch_q8_decode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream);

}  // namespace zs
