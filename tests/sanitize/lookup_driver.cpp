// The kernels' own look-up of a workgroup's tile (find_tensor, tile_in_runs) on
// the tables that the entry points fill, on the host under AddressSanitizer and
// UndefinedBehaviorSanitizer: over the launches of a call every tile of every
// tensor is taken by one workgroup (run by tests/test_tensors_lookup.py).
// Addresses are made up and never used.
#include <cstdio>
#include <vector>

#include "../../fsdp_sharded_optimizer_amd/csrc/api_tensors.hip"

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            std::fprintf(stderr, "line %d: check failed: %s\n", __LINE__, #cond); \
            std::exit(1);                                                         \
        }                                                                         \
    } while (0)

namespace {

int64_t tiles_seen, runs_launches;

// every workgroup's tile, once each, and the tensor it is in; `record` is called with
// each tensor of the table that has tiles, and their number, in order
template <int N, typename Record>
void replay(const ListTable<N>& tab, int64_t tiles, bool runs, Record record) {
    std::vector<int64_t> of((size_t)tiles, -1), first((size_t)tiles, 0);
    for (int64_t w = 0; w < tiles; ++w) {
        const uint32_t tile = runs ? tile_in_runs((uint32_t)w, (uint32_t)tiles) : (uint32_t)w;
        CHECK(tile < (uint64_t)tiles && of[tile] < 0);
        uint32_t from = kNoTile;
        of[tile] = find_tensor(tab, tile, from);
        CHECK(of[tile] < N && from <= tile && tab.start[of[tile] + 1] > tile);
        first[tile] = from;
    }
    for (int64_t a = 0, b; a < tiles; a = b) {
        CHECK(first[a] == a);
        for (b = a; b < tiles && of[b] == of[a]; ++b) CHECK(first[b] == a);
        record((uint32_t)of[a], b - a);
    }
    tiles_seen += tiles;
    runs_launches += runs;
}

std::vector<int64_t> lengths;   // of the list under test, in tiles
size_t at;                      // the list's next tensor
void next_tensor(int64_t n) {
    while (at < lengths.size() && lengths[at] == 0) ++at;
    CHECK(at < lengths.size() && lengths[at] == n);
    ++at;
}

hipError_t q8_launch(const Q8Batch& b, int64_t tiles) {
    replay(b.tab, tiles, b.runs != 0, [&](uint32_t t, int64_t n) {
        CHECK((size_t)b.index + t < lengths.size() && lengths[b.index + t] == n);
        next_tensor(n);
        CHECK(at == (size_t)b.index + t + 1);
    });
    return hipSuccess;
}

}  // namespace

namespace zs {

int64_t norm_tile_elems(int bf16) { return bf16 ? 8192 : 4096; }
hipError_t launch_norm_tensors(const NormBatch& b, int, bool, int64_t tiles, float, double*, hipStream_t) {
    replay(b.tab, tiles, false, [](uint32_t, int64_t n) { next_tensor(n); });
    return hipSuccess;
}
hipError_t launch_list_sum(const double*, int64_t, double*, double*, hipStream_t) { return hipSuccess; }
hipError_t launch_adamw_tensors(const AdamwBatch& b, int, int, bool, bool, int64_t tiles, hipStream_t) {
    replay(b.tab, tiles, false, [](uint32_t, int64_t n) { next_tensor(n); });
    return hipSuccess;
}
hipError_t launch_adamw_q8(const Q8Batch& b, int, int, bool, int64_t tiles, hipStream_t) { return q8_launch(b, tiles); }
hipError_t launch_q8_encode(const Q8Batch& b, int, int64_t tiles, hipStream_t) { return q8_launch(b, tiles); }
hipError_t launch_q8_decode(const Q8Batch& b, int, int64_t tiles, hipStream_t) { return q8_launch(b, tiles); }

}  // namespace zs

extern "C" int32_t adamw_scalars(const zs_adamw*, zs_adamw_scalars* out) {
    std::memset(out, 0, sizeof(*out));
    return ZS_OK;
}

namespace {

void* fake(uint64_t x) { return reinterpret_cast<void*>((uintptr_t)(0x700000000000u + x)); }

template <typename Call>
void over_tiles(const std::vector<int64_t>& numels, int64_t tile, Call call) {
    lengths.clear();
    for (int64_t n : numels) lengths.push_back((n + tile - 1) / tile);
    at = 0;
    CHECK(call() == ZS_OK);
    while (at < lengths.size() && lengths[at] == 0) ++at;
    CHECK(at == lengths.size());
}

// off: bytes that the streams start off their cache lines
void calls(const std::vector<int64_t>& numels, uint64_t off) {
    const int32_t count = (int32_t)numels.size();
    std::vector<zs_adamw_tensor> step;
    std::vector<zs_adamw_q8_tensor> q8;
    std::vector<zs_moments_q8> mom;
    std::vector<zs_tensor> grads((size_t)count);
    zs_adamw hp{};
    hp.step = 1, hp.lr = 1e-3, hp.beta1 = 0.9, hp.beta2 = 0.95, hp.eps = 1e-8, hp.grad_scale = 1.0;
    const uint64_t each = uint64_t(1) << 20, kind = each * 2048;
    for (int32_t k = 0; k < count; ++k) {
        const int64_t n = numels[(size_t)k];
        CHECK(n * 4 + 64 < (int64_t)each);
        const uint64_t a = each * (uint64_t)k;
        // the fp32 step's moments start on a whole tile, so its tiles are the tensor's own
        step.push_back({fake(a + off), fake(kind + a + off), static_cast<float*>(fake(2 * kind + a)),
                        static_cast<float*>(fake(3 * kind + a)), nullptr, n});
        q8.push_back({fake(a + off), fake(kind + a + off), fake(2 * kind + a), nullptr, n});
        mom.push_back({fake(a + off), fake(kind + a + off), fake(2 * kind + a), n});
        grads[(size_t)k].ptr = fake(a + off), grads[(size_t)k].numel = n;
    }
    over_tiles(numels, kListTile,
               [&] { return adamw_step_tensors(&hp, step.data(), count, ZS_F32, ZS_F32, nullptr, nullptr); });
    over_tiles(numels, kQ8Pad,
               [&] { return adamw_step_tensors_q8(&hp, 1, q8.data(), count, ZS_F32, ZS_F32, nullptr, nullptr); });
    over_tiles(numels, kQ8Pad, [&] { return moments_q8_encode(mom.data(), count, ZS_F32, 1, nullptr); });
    const int64_t before = runs_launches;
    over_tiles(numels, kQ8Pad, [&] { return moments_q8_decode(mom.data(), count, ZS_F32, nullptr); });
    CHECK(tiles_seen == 0 || (runs_launches > before) == (off != 0) || count == 0);
    const int64_t need = grad_norm_sq_tensors_workspace_bytes(grads.data(), count, ZS_F32);
    over_tiles(numels, 4096, [&] {
        return grad_norm_sq_tensors(grads.data(), count, ZS_F32, 1.0, reinterpret_cast<double*>(0x100000),
                                    reinterpret_cast<void*>(0x200000), need, nullptr);
    });
}

}  // namespace

int main() {
    for (uint32_t n = 1; n < 2000; ++n) {   // the runs of tiles alone: each tile once, a whole 32 by fours per XCD
        std::vector<char> seen(n, 0);
        for (uint32_t w = 0; w < n; ++w) {
            const uint32_t t = tile_in_runs(w, n);
            CHECK(t < n && !seen[t] && t / 32 == w / 32);
            if (w % 32 >= 8 && w / 32 * 32 + 32 <= n) CHECK(t == tile_in_runs(w - 8, n) + 1);
            seen[t] = 1;
        }
    }
    uint32_t rng = 99;
    for (int count : {1, 2, 7, 8, 9, 97, 98, 99, 149, 150, 151, 300, 327, 328, 329, 700})
        for (int kind = 0; kind < 4; ++kind)
            for (uint64_t off : {0, 4}) {
                std::vector<int64_t> numels;
                for (int k = 0; k < count; ++k) {
                    rng = rng * 1664525u + 1013904223u;
                    const int64_t r = rng >> 8;
                    numels.push_back(kind == 0   ? 1 + r % 300
                                     : kind == 1 ? (r % 3 == 0 ? 0 : 1 + r % 5000)
                                     : kind == 2 ? (r % 16 == 0 ? 100000 + r % 100000 : 1 + r % 3)
                                                 : 512 * (1 + r % 9));
                }
                numels[0] += numels[0] == 0;
                calls(numels, off);
            }
    std::printf("look-up: ok, %lld tiles, %lld launches in runs\n", (long long)tiles_seen, (long long)runs_launches);
    return 0;
}
