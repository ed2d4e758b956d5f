// AdamW over a list of tensors with fp32 moments.
//
// The update of one element is adamw.hip's (adamw_math.h: the same operations
// and roundings, so a tensor gets the bits adamw_step or adamw_step_no_master
// would give it); here one launch covers up to 98 tensors of any sizes.
// HBM-bound: with fp32 parameters 24 B/element of parameter and moments plus
// the gradient (2 or 4) and the bf16 re-cast (2); with bf16 parameters 20 plus
// the gradient.
//
// Layout: the flat step's: one-wave workgroups of 256 elements, 4 consecutive
// per lane, a 128-bit access per fp32 stream (64-bit per bf16 one), residency
// capped by reserved LDS.  A workgroup's tile lies in one tensor (find_tensor).
#include "adamw_math.h"
#include "tensors.h"

namespace zs {
namespace {

constexpr int kWave = 64;
// LDS reserved (never touched) per workgroup, to cap how many share a CU (too
// many keep too many DRAM rows open): the cap that keeps about 80 KiB in flight
// per CU.  Measured, % of the 8 TB/s peak uncapped and at 8 / 10 / 12 / 13 / 14 / 16
// KiB: fp32 parameters with re-casts, fp32 gradients (634M) 76.5, 79.9 / 80.7 /
// 81.8 / 82.8 / 83.1 / 81.5, bf16 gradients (809M) 75.4, 79.2 / 79.9 / 81.1 / 82.7 /
// 82.1 / 79.1; bf16 parameters, fp32 gradients (855M) 78.5, 81.3 / 81.2 / 82.2 /
// 80.8 / 78.2 / 74.4, bf16 gradients (855M) 78.0, 81.1 / 81.5 / 80.6 / 77.9 / 74.3 /
// 70.1.  A launch of less than 8M elements is not long enough for that: one tensor
// of 2M / 8M / 32M / 64M elements, us uncapped and capped, fp32 parameters and
// gradients 12.7, 13.6 / 40.6, 40.6 / 143, 142 / 318, 291; bf16 gradients 12.8,
// 13.5 / 38.5, 36.8 / 139, 133 / 277, 263; bf16 parameters and gradients 10.8, 11.2 /
// 30.0, 29.0 / 106, 102 / 208, 203.  (bf16 parameters with fp32 gradients are 4-7 %
// faster uncapped up to 48M, 11.4, 11.6 / 33.1, 34.4 / 112, 118, and 4 % slower at
// 64M, 241, 232.)
template <bool PBF16, bool GBF16>
constexpr unsigned kLds = PBF16 ? (GBF16 ? 10240 : 12288) : (GBF16 ? 13312 : 14336);
// Where most tiles start off a cache line in some stream, their gradients are
// kept (neighbours share lines of them) and one KiB more is reserved.  405M, us
// without either / with the first / with both: fp32 parameters with re-casts, every
// stream at an offset of its own 2159 / 2120 / 2079, the re-casts alone 1766 / 1773 /
// 1759; bf16 gradients alone (bf16 parameters) 1395 / 1360 / 1337; fp32 gradients
// alone 1834 / 1809 / 1808.
constexpr unsigned kOffLineLds = 1024;
constexpr int64_t kCapTiles = 32768;

template <bool PBF16, bool GBF16, bool DEV, bool KEEP>
__global__ __launch_bounds__(kWave) void adamw_tensors_kernel(const AdamwBatch b) {
    using P = typename GradType<PBF16>::T;
    using G = typename GradType<GBF16>::T;
    uint32_t first;
    const AdamwEntry e = b.e[find_tensor(b.tab, blockIdx.x, first)];
    const AdamwScalars sc = DEV ? *b.sc_dev : b.sc;
    P* const param = unpack_ptr<P>(e.lo[0], e.hi[0]);
    const G* const grad = unpack_ptr<const G>(e.lo[1], e.hi[0] >> 16);
    float* const exp_avg = unpack_ptr<float>(e.lo[2], e.hi[1]);
    float* const exp_avg_sq = unpack_ptr<float>(e.lo[3], e.hi[1] >> 16);
    uint16_t* const copy = unpack_ptr<uint16_t>(e.lo[4], e.hi[2]);
    const int64_t n = e.numel;
    const int64_t i = (int64_t)(blockIdx.x - first) * kListTile - (e.hi[2] >> 16) + threadIdx.x * 4;
    float coef;
    if (i >= 0 && i + 4 <= n) {
        // the loads are issued before the clip coefficient is resolved
        const f32x4 g4 = ld4<KEEP>(grad + i);
        f32x4 p4 = ld4(param + i);
        f32x4 m4 = ld4(exp_avg + i);
        f32x4 v4 = ld4(exp_avg_sq + i);
        if (!clip_coef(sc, b.norm_sq, coef)) return;
        float gs[4] = {g4.x, g4.y, g4.z, g4.w};
        float ps[4] = {p4.x, p4.y, p4.z, p4.w};
        float ms[4] = {m4.x, m4.y, m4.z, m4.w};
        float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = adam_elem(sc, coef, gs[j], ms[j], vs[j]);
            ps[j] = apply_step(sc, ps[j], u);
        }
        const f32x4 po = {ps[0], ps[1], ps[2], ps[3]};
        st4(param + i, po);
        st4(exp_avg + i, f32x4{ms[0], ms[1], ms[2], ms[3]});
        st4(exp_avg_sq + i, f32x4{vs[0], vs[1], vs[2], vs[3]});
        if (!PBF16 && copy != nullptr) st4(copy + i, po);
        return;
    }
    // lanes across a tensor's start or end (or outside it)
    if (!clip_coef(sc, b.norm_sq, coef)) return;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const int64_t k = i + j;
        if (k < 0 || k >= n) continue;
        float m = exp_avg[k], v = exp_avg_sq[k];
        const float u = adam_elem(sc, coef, widen(grad[k]), m, v);
        const float p = apply_step(sc, widen(param[k]), u);
        st1(param + k, p);
        exp_avg[k] = m;
        exp_avg_sq[k] = v;
        if (!PBF16 && copy != nullptr) st1(copy + k, p);
    }
}

template <bool PBF16, bool GBF16>
hipError_t launch(const AdamwBatch& b, bool keep, bool off_line, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    const unsigned lds = tiles < kCapTiles ? 0 : kLds<PBF16, GBF16> + (off_line ? kOffLineLds : 0);
    const auto kernel =
        b.sc_dev != nullptr
            ? (keep ? adamw_tensors_kernel<PBF16, GBF16, true, true> : adamw_tensors_kernel<PBF16, GBF16, true, false>)
            : (keep ? adamw_tensors_kernel<PBF16, GBF16, false, true> : adamw_tensors_kernel<PBF16, GBF16, false, false>);
    hipLaunchKernelGGL(kernel, grid, block, lds, stream, b);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw_tensors(const AdamwBatch& b, int param_bf16, int grad_bf16, bool keep, bool off_line,
                                int64_t tiles, hipStream_t stream) {
    const auto run = param_bf16 ? (grad_bf16 ? launch<true, true> : launch<true, false>)
                                : (grad_bf16 ? launch<false, true> : launch<false, false>);
    return run(b, keep, off_line, tiles, stream);
}

}  // namespace zs
