// The tile sizes that the calls over matrices launch with, asked of the entry
// points' source on the host (run by tests/test_matrices_tile_sizes.py).  A line of
// input is one call; a line of output the sides of its launches' tiles.
//   product|gram dtype m n k count        (gram: m x k, n is not looked at)
//   muon rows cols count                  -> of S and its polynomial, of X, of the last X
#include <cstdio>
#include <cstring>
#include <set>
#include <vector>

#include "../../fsdp_sharded_optimizer_amd/csrc/api_matrices.hip"

namespace zs {
thread_local int32_t g_last_hip_error = 0;
std::set<int64_t> products_of, phase_of[3], final_of;

hipError_t launch_products(const ProductBatch&, int size, bool, bool, bool, int64_t, hipStream_t) {
    products_of.insert(tile_side(size));
    return hipSuccess;
}
hipError_t launch_ns(const NsBatch&, int phase, int size, int64_t, hipStream_t) {
    phase_of[phase].insert(tile_side(size));
    return hipSuccess;
}
hipError_t launch_ns_final(const FinalBatch&, int, int size, bool, int64_t, hipStream_t) {
    final_of.insert(tile_side(size));
    return hipSuccess;
}
hipError_t launch_stage(const StageBatch&, int, int, bool, bool, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_momentum(const MomentumBatch&, int, bool, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_inverse_norms(const NormsBatch&, hipStream_t) { return hipSuccess; }
hipError_t launch_pack(const PackBatch&, int, bool, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_skinny_gram(const NsBatch&, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_skinny_steps(const NsBatch&, int64_t, hipStream_t) { return hipSuccess; }
}  // namespace zs

int main() {
    uint64_t place = 0;
    auto fresh = [&](int64_t bytes) {   // made up, never followed
        const uint64_t p = place;
        place += (uint64_t)(bytes + 511) / 256 * 256;
        return reinterpret_cast<void*>(p);
    };
    char kind[16];
    while (std::scanf("%15s", kind) == 1) {
        place = uint64_t(0x1000) << 32;
        products_of.clear(), final_of.clear();
        for (auto& s : phase_of) s.clear();
        void* const ws = reinterpret_cast<void*>(uint64_t(0x5000) << 32);
        int32_t rc;
        if (std::strcmp(kind, "muon") == 0) {
            long long rows, cols, count;
            if (std::scanf("%lld %lld %lld", &rows, &cols, &count) != 3) return 1;
            std::vector<zs_muon_matrix> list((size_t)count);
            for (auto& x : list)
                x = zs_muon_matrix{fresh(rows * cols * 4), fresh(rows * cols * 4), static_cast<float*>(fresh(rows * cols * 4)),
                                   nullptr, rows, cols, 1.0};
            const zs_muon hp = {0.01, 0.9, 0.1, 3.4445, -4.775, 2.0315, 1e-7, 1.0, 0.0, 0.0, 1, 5};
            rc = muon_step_matrices(&hp, list.data(), (int32_t)count, ZS_F32, ZS_BF16, nullptr, ws,
                                    muon_step_matrices_workspace_bytes(list.data(), (int32_t)count), nullptr);
        } else {
            long long m, n, k, count;
            int dtype;
            if (std::scanf("%d %lld %lld %lld %lld", &dtype, &m, &n, &k, &count) != 5) return 1;
            if (std::strcmp(kind, "gram") == 0) {
                std::vector<zs_gram> list((size_t)count);
                for (auto& x : list) x = zs_gram{fresh(m * k * 4), nullptr, fresh(m * m * 4), m, k, 0, 0};
                rc = gram_add_matrices(list.data(), (int32_t)count, dtype, ZS_F32, 1.0, 0.0, ws,
                                       gram_add_matrices_workspace_bytes(list.data(), (int32_t)count, dtype), nullptr);
            } else {
                std::vector<zs_product> list((size_t)count);
                for (auto& x : list) x = zs_product{fresh(m * k * 4), fresh(k * n * 4), nullptr, fresh(m * n * 4), m, n, k};
                rc = product_add_matrices(list.data(), (int32_t)count, dtype, ZS_F32, ZS_F32, 0, 1.0, 0.0, ws,
                                          product_add_matrices_workspace_bytes(list.data(), (int32_t)count, dtype, 0), nullptr);
            }
        }
        if (rc != ZS_OK) return 2;
        for (const auto* of : {&products_of, &phase_of[kNsGram], &phase_of[kNsPoly], &phase_of[kNsUpdate], &final_of})
            for (int64_t side : *of) std::printf("%lld ", (long long)side);
        std::printf("\n");
    }
    return 0;
}
