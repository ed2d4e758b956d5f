// Drives the host side of the calls over lists of tensors under
// AddressSanitizer and UndefinedBehaviorSanitizer (built with hipcc, the
// sanitizers on the host pass only; run by tests/test_tensors_sanitizers.py on
// a machine without a GPU).  Lists are allocated at their exact sizes.  Valid
// calls are made as well: without a GPU their first launch fails, after every
// check and after the launch's table has been filled, so the whole host path
// runs; no pointer is dereferenced.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../include/zshard_tensors.h"
#include "../../fsdp_sharded_optimizer_amd/csrc/tensors.h"

#define CHECK(cond)                                                              \
    do {                                                                         \
        if (!(cond)) {                                                           \
            std::fprintf(stderr, "line %d: check failed: %s\n", __LINE__, #cond); \
            return 1;                                                            \
        }                                                                        \
    } while (0)

static const uintptr_t FAKE = 0x7F0000000000ull;
static void* fake(uint64_t off) { return reinterpret_cast<void*>(FAKE + off); }
template <typename T>
static T* fake_as(uint64_t off) { return reinterpret_cast<T*>(FAKE + off); }

// find_tensor's scan, on the host, for a table as the entry points fill it
template <int N>
static int find(const zs::ListTable<N>& tab, uint32_t w) {
    const uint32_t part = w >> tab.shift;
    if (part >= (uint32_t)zs::kListBuckets) return -1;
    uint32_t t = tab.bucket[part >> 2] >> (8 * (part & 3)) & 0xFFu, from;
    do {
        from = t;
        if (from + zs::kListScan >= N + zs::kListScan) return -2;
        for (int k = 1; k <= zs::kListScan; ++k) t += w >= tab.start[from + k] ? 1 : 0;
    } while (t == from + zs::kListScan);
    return (int)t;
}

// the runs of tiles are a permutation of the workgroups
static int check_runs() {
    for (uint32_t n = 1; n < 300; ++n) {
        std::vector<unsigned char> seen(n, 0);
        for (uint32_t w = 0; w < n; ++w) {
            const uint32_t base = w / 32 * 32, i = w % 32;
            const uint32_t t = base + 32 > n ? w : base + (i % 8) * 4 + i / 8;
            if (t >= n || seen[t]) return 1;
            seen[t] = 1;
        }
    }
    return 0;
}

// a table built as the entry points build theirs finds every workgroup's tensor
static int check_tables() {
    uint32_t rng = 1;
    for (int round = 0; round < 400; ++round) {
        zs::ListTable<98> tab;
        const int count = 1 + (int)(rng % 98);
        std::vector<uint32_t> tiles;
        uint64_t total = 0;
        for (auto& s : tab.start) s = zs::kNoTile;
        for (int k = 0; k < count; ++k) {
            rng = rng * 1664525u + 1013904223u;
            const uint32_t n = (rng >> 8) % 5 == 0 ? 1 + (rng >> 12) % 3000 : 1 + (rng >> 12) % 2;
            tab.start[k] = (uint32_t)total;
            total += n;
            tiles.push_back(n);
        }
        tab.shift = 0;
        while (((total - 1) >> tab.shift) >= (uint64_t)zs::kListBuckets) ++tab.shift;
        for (auto& b : tab.bucket) b = 0;
        int t = 0;
        for (int part = 0; part < zs::kListBuckets && ((uint64_t)part << tab.shift) < total; ++part) {
            while (tab.start[t + 1] <= ((uint64_t)part << tab.shift)) ++t;
            tab.bucket[part / 4] |= (uint32_t)t << (8 * (part % 4));
        }
        uint32_t w = 0;
        for (int k = 0; k < count; ++k)
            for (uint32_t i = 0; i < tiles[k]; ++i, ++w)
                if (find(tab, w) != k) return 1;
    }
    return 0;
}

int main() {
    CHECK(check_runs() == 0);
    CHECK(check_tables() == 0);
    zs_adamw hp = {};
    hp.lr = 1e-3, hp.beta1 = 0.9, hp.beta2 = 0.95, hp.eps = 1e-8, hp.grad_scale = 1.0, hp.max_norm = 1.0, hp.step = 1;
    const int32_t counts[] = {1, 2, 97, 98, 99, 240, 241, 1500};
    for (int32_t count : counts) {
        // ascending, descending and scattered buffers, some tensors empty, one of more than 2^31 elements
        for (int order = 0; order < 3; ++order) {
            std::vector<zs_adamw_tensor> step((size_t)count);
            std::vector<zs_adamw_q8_tensor> q8((size_t)count);
            std::vector<zs_moments_q8> mom((size_t)count);
            std::vector<zs_tensor> grads((size_t)count);
            const uint64_t each = 1ull << 16;
            for (int32_t k = 0; k < count; ++k) {
                const uint64_t at = order == 0 ? (uint64_t)k : order == 1 ? (uint64_t)(count - 1 - k) : (uint64_t)(k * 7919ll % count);
                const int64_t n = k % 5 == 3 ? 0 : 1 + (k * 37) % 900;
                const uint64_t base = at * each * 6, odd = order == 2 ? 4 : 0;
                step[k] = {fake(base + odd), fake(base + each + odd), fake_as<float>(base + 2 * each + odd),
                           fake_as<float>(base + 3 * each + odd), fake_as<uint16_t>(base + 4 * each + 2), n};
                q8[k] = {fake(base + odd), fake(base + each), fake(base + 2 * each), k % 2 ? nullptr : fake_as<uint16_t>(base + 3 * each + 2), n};
                mom[k] = {fake(base), k % 3 ? fake(base + each) : nullptr, fake(base + 2 * each), n};
                grads[k] = {fake(base), n};
            }
            CHECK(adamw_step_tensors(&hp, step.data(), count, ZS_F32, ZS_F32, nullptr, nullptr) == ZS_EHIP);
            CHECK(adamw_step_tensors_dev(fake_as<zs_adamw_scalars>(1ull << 40), step.data(), count, ZS_F32, ZS_BF16,
                                         fake_as<double>(1ull << 41), nullptr) == ZS_EHIP);
            CHECK(adamw_step_tensors_q8(&hp, 7u, q8.data(), count, ZS_F32, ZS_BF16, nullptr, nullptr) == ZS_EHIP);
            CHECK(moments_q8_encode(mom.data(), count, ZS_BF16, 1u, nullptr) == ZS_EHIP);
            CHECK(moments_q8_decode(mom.data(), count, ZS_F32, nullptr) == ZS_EHIP);
            const int64_t need = grad_norm_sq_tensors_workspace_bytes(grads.data(), count, ZS_F32);
            CHECK(need > 0);
            CHECK(grad_norm_sq_tensors(grads.data(), count, ZS_F32, 0.5, fake_as<double>(1ull << 40), fake(1ull << 41),
                                       need, nullptr) == ZS_EHIP);
            // one tensor's parameter inside another's second moments
            const int32_t last = count - 1;
            if (count > 4 && step[last].numel > 0) {
                zs_adamw_tensor keep = step[0];
                step[0].param = reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(step[last].exp_avg_sq) + 4);
                step[0].numel = 1;
                CHECK(step[last].numel < 2 ||
                      adamw_step_tensors(&hp, step.data(), count, ZS_F32, ZS_F32, nullptr, nullptr) == ZS_EOVERLAP);
                step[0] = keep;
            }
        }
    }
    // a tensor of several entries, the most elements a call takes, and one more
    zs_adamw_tensor huge = {fake(0), fake(1ull << 42), fake_as<float>(1ull << 43), fake_as<float>(3ull << 42), nullptr, 1ll << 39};
    CHECK(adamw_step_tensors(&hp, &huge, 1, ZS_BF16, ZS_BF16, nullptr, nullptr) == ZS_EHIP);
    zs_adamw_q8_tensor huge8 = {fake(0), fake(1ull << 42), fake(1ull << 43), nullptr, 1ll << 39};
    CHECK(adamw_step_tensors_q8(&hp, 0u, &huge8, 1, ZS_BF16, ZS_BF16, nullptr, nullptr) == ZS_EHIP);
    huge.numel += 1;
    CHECK(adamw_step_tensors(&hp, &huge, 1, ZS_BF16, ZS_BF16, nullptr, nullptr) == ZS_EINVAL);
    // an address that 48 bits do not hold
    huge.numel = 4;
    huge.param = reinterpret_cast<void*>(1ull << 52);
    CHECK(adamw_step_tensors(&hp, &huge, 1, ZS_BF16, ZS_BF16, nullptr, nullptr) == ZS_EINVAL);
    zs_tensor far = {reinterpret_cast<void*>(1ull << 52), 4};
    CHECK(grad_norm_sq_tensors(&far, 1, ZS_F32, 1.0, fake_as<double>(0), fake(64), 64, nullptr) == ZS_EINVAL);
    std::printf("tensors sanitizer drive: ok\n");
    return 0;
}
