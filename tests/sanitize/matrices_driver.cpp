// The tables that the calls over lists of matrices and of mixed precision launch
// with, replayed on the host under AddressSanitizer and UndefinedBehaviorSanitizer:
// the entry points' source with launches that look every workgroup up as the
// kernels do and check what it would read and write: every tile of every matrix
// once, every place in the workspace inside it and a matrix's own (run by
// tests/test_matrices_tables.py).  Addresses are made up and never used.
#include <cstdio>
#include <map>
#include <random>
#include <vector>

#include "../../fsdp_sharded_optimizer_amd/csrc/api_clip.hip"
#include "../../fsdp_sharded_optimizer_amd/csrc/api_matrices.hip"

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            std::fprintf(stderr, "line %d: check failed: %s\n", __LINE__, #cond); \
            std::exit(1);                                                         \
        }                                                                         \
    } while (0)

namespace zs {
thread_local int32_t g_last_hip_error = 0;
int64_t mixed_tile_elems(int bf16) { return bf16 ? 8192 : 4096; }
}  // namespace zs

namespace {

constexpr uint64_t kWs = uint64_t(0x5000) << 32;   // the workspace
int64_t ws_bytes;

template <int N>
uint32_t find(const ListTable<N>& tab, uint32_t w, uint32_t& first) {
    const uint32_t t = find_tensor(tab, w, first);
    CHECK(t < (uint32_t)N && first <= w && w < tab.start[t + 1]);
    return t;
}
uint64_t address(uint32_t lo, uint32_t hi16) { return (uint64_t)(hi16 & 0xFFFFu) << 32 | lo; }
int64_t tiles_of(int64_t m, int64_t n, int size, bool triangle) {
    const int64_t s = tile_side(size), r = (m + s - 1) / s;
    return triangle ? r * (r + 1) / 2 : r * ((n + s - 1) / s);
}
void inside(uint64_t p, int64_t bytes) { CHECK(p >= kWs && p % 8 == 0 && (int64_t)(p - kWs) + bytes <= ws_bytes); }

// what the launches of one call have been seen to do
std::map<uint64_t, int64_t> seen[8];   // by kind: a destination's address -> workgroups
std::map<uint64_t, uint64_t> taken;    // pieces of the workspace of the group under way
int64_t launches, partials_seen, clip_elems;

void take(uint64_t from, int64_t bytes) {
    inside(from, bytes);
    auto next = taken.lower_bound(from + 1);
    if (next != taken.begin()) CHECK(std::prev(next)->second <= from || std::prev(next)->first == from);
    if (next != taken.end()) CHECK(from + (uint64_t)bytes <= next->first);
    taken[from] = from + (uint64_t)bytes;
}

}  // namespace

namespace zs {

hipError_t launch_products(const ProductBatch& b, int size, bool b_cols, bool sym, bool, int64_t tiles, hipStream_t) {
    ++launches;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const ProductEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        CHECK(w - first < tiles_of(e.m, e.n, size, sym));
        ++seen[0][address(e.lo[3], e.hi[1] >> 16)];
        if (e.k_tiles == 0 || w != first) continue;
        const uint64_t a = address(e.lo[0], e.hi[0]), o = address(e.lo[1], e.hi[0] >> 16);
        CHECK(a % 16 == 0 && o % 16 == 0 && e.lda >= e.k_tiles * 64 && e.lda % 8 == 0 && e.ldb % 8 == 0);
        CHECK(b_cols ? e.ldb >= e.n : e.ldb >= e.k_tiles * 64);
        // what is read from the workspace was copied there
        CHECK((a < kWs || taken.count(a) == 1) && (o < kWs || taken.count(o) == 1));
        if (a >= kWs) inside(a, ((int64_t)e.m - 1) * e.lda * 2 + e.k_tiles * 128);
        if (o >= kWs) inside(o, b_cols ? (int64_t)e.k_tiles * 64 * e.ldb * 2 : ((int64_t)e.n - 1) * e.ldb * 2 + e.k_tiles * 128);
    }
    return hipSuccess;
}

hipError_t launch_stage(const StageBatch& b, int src_bf16, int kind, bool, bool, int64_t tiles, hipStream_t) {
    ++launches;
    CHECK((kind == kStagePlain) == (src_bf16 != 0));
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const StageEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        CHECK(w - first < stage_tiles(e.rows, e.cols));
        if (w == first) take(address(e.lo[1], e.hi >> 16), pad_side(e.rows) * pad_side(e.cols) * 2 * (kind == kStagePlain ? 1 : 3));
    }
    return hipSuccess;
}

hipError_t launch_momentum(const MomentumBatch& b, int, bool, int64_t tiles, hipStream_t) {
    ++launches;
    inside((uint64_t)(uintptr_t)b.partials, tiles * 8);
    partials_seen += tiles;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const MomentumEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        CHECK((w - first) * kMomentumTile < (int64_t)e.numel);
        ++seen[1][address(e.lo[0], e.hi)];
    }
    return hipSuccess;
}

hipError_t launch_inverse_norms(const NormsBatch& b, hipStream_t) {
    ++launches;
    CHECK(b.count >= 1 && b.count <= 960);
    for (uint32_t k = 0; k < b.count; ++k) CHECK(b.start[k] < b.start[k + 1]);
    inside((uint64_t)(uintptr_t)(b.partials + b.start[0]), (int64_t)(b.start[b.count] - b.start[0]) * 8);
    const uint64_t at = (uint64_t)(uintptr_t)b.inverse;
    CHECK(at >= kWs && (int64_t)(at - kWs) + b.count * 4 <= ws_bytes);
    partials_seen -= b.start[b.count] - b.start[0];
    return hipSuccess;
}

hipError_t launch_pack(const PackBatch& b, int, bool, int64_t tiles, hipStream_t) {
    ++launches;
    CHECK(b.ws == reinterpret_cast<char*>(kWs));
    uint32_t most = 0;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const uint32_t t = find(b.tab, (uint32_t)w, first);
        const PackEntry& e = b.e[t];
        const int64_t m = e.m, n = e.n & ~kTall;
        CHECK(m <= n && w - first < stage_tiles(m, n));
        if (w == first) take(kWs + (uint64_t)e.base * kNsUnit, ns_bytes(m, n));
        most = std::max(most, t);
        ++seen[2][address(e.lo[0], e.hi)];
    }
    const uint64_t at = b.inverse != nullptr ? (uint64_t)(uintptr_t)b.inverse : (uint64_t)(uintptr_t)b.partials;
    if (b.inverse != nullptr) {
        CHECK(at >= kWs && (int64_t)(at - kWs) + (most + 1) * 4 <= ws_bytes);
    } else {   // from each matrix's partials, which follow one another in the table's order
        int64_t next = b.e[0].partial;
        for (uint32_t t = 0; t <= most; ++t) {
            const int64_t n = ((int64_t)b.e[t].m * (b.e[t].n & ~kTall) + kMomentumTile - 1) / kMomentumTile;
            CHECK(n <= kPackPartials && b.e[t].partial == next);
            next += n;
            partials_seen -= n;
        }
        inside((uint64_t)(uintptr_t)(b.partials + b.e[0].partial), (next - b.e[0].partial) * 8);
    }
    for (const auto& piece : taken) CHECK(piece.second <= at);   // the norms lie behind the matrices
    return hipSuccess;
}

hipError_t launch_ns(const NsBatch& b, int phase, int size, int64_t tiles, hipStream_t) {
    ++launches;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const NsEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        CHECK(e.m > kSkinny && w - first < tiles_of(pad_side(e.m), pad_side(e.n), size, phase != kNsUpdate));
        CHECK(taken.count(kWs + (uint64_t)e.base * kNsUnit) == 1);
        ++seen[3 + (phase == kNsUpdate)][kWs + (uint64_t)e.base * kNsUnit];
    }
    return hipSuccess;
}
hipError_t launch_skinny_gram(const NsBatch& b, int64_t tiles, hipStream_t) {
    ++launches;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const NsEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        const SkinnyPlace p(e.n);
        CHECK(e.m <= kSkinny && (w - first) * p.chunk < p.np / 64 && p.parts() + p.chunks * SkinnyPlace::kPart <= p.q());
    }
    return hipSuccess;
}
hipError_t launch_skinny_steps(const NsBatch& b, int64_t count, hipStream_t) {
    ++launches;
    for (int64_t w = 0; w < count; ++w) {   // an entry each
        uint32_t first;
        CHECK(find(b.tab, (uint32_t)w, first) == (uint32_t)w && b.steps >= 1);
    }
    return hipSuccess;
}
hipError_t launch_ns_final(const FinalBatch& b, int, int size, bool skinny, int64_t tiles, hipStream_t) {
    ++launches;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const FinalEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        CHECK((e.m <= kSkinny) == skinny && w - first < tiles_of(e.m, e.n & ~kTall, size, false));
        CHECK(taken.count(kWs + (uint64_t)e.base * kNsUnit) == 1);
        ++seen[5][address(e.lo[0], e.hi)];
    }
    // the last launch of a group: the next one has the workspace anew
    return hipSuccess;
}

hipError_t launch_norms(const NormBatch& b, bool, int64_t tiles, float, double* partials, hipStream_t) {
    ++launches;
    inside((uint64_t)(uintptr_t)partials, tiles * 8);
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const NormEntry& e = b.e[find(b.tab, (uint32_t)w, first)];
        ++seen[6][address(e.lo, e.hi_tail)];
    }
    partials_seen += tiles;
    return hipSuccess;
}
hipError_t launch_tensor_sums(const TensorSums& b, hipStream_t) {
    ++launches;
    CHECK(b.count >= 1 && b.count <= (uint32_t)kSumsMax);
    for (uint32_t k = 0; k < b.count; ++k) CHECK(b.start[k] <= b.start[k + 1]);
    CHECK(b.start[0] == 0 && b.start[b.count] == b.grid);
    partials_seen -= b.grid;
    return hipSuccess;
}
hipError_t launch_few_sums(const TensorSums& b, double*, hipStream_t s) {
    CHECK(b.count <= (uint32_t)kFewTensors);
    return launch_tensor_sums(b, s);
}
hipError_t launch_total(const double*, int64_t, double*, hipStream_t) {
    ++launches;
    return hipSuccess;
}
hipError_t launch_clip(const ClipBatch& b, int64_t tiles, hipStream_t) {
    ++launches;
    for (int64_t w = 0; w < tiles; ++w) {
        uint32_t first;
        const uint32_t t = find(b.tab, (uint32_t)w, first);
        const int64_t n = (int64_t)b.e[t].numel_less_1 + 1, at = (w - first) * kClipTile;
        CHECK(at < n);
        clip_elems += std::min(kClipTile, n - at);
        CHECK((b.bf16[t / 16] >> (2 * (t % 16)) & 3u) == (uint32_t)(b.e[t].lo[0] >> 4 & 3u));   // made up so below
    }
    return hipSuccess;
}

}  // namespace zs

namespace {

std::mt19937_64 rng(7);
int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }
uint64_t place_at;
void* fresh(int64_t bytes, int off) {   // a buffer of its own, `off` bytes past a boundary of 1 KiB
    const uint64_t p = place_at + (uint64_t)off;
    place_at += (uint64_t)(bytes + 2047) / 1024 * 1024;
    return reinterpret_cast<void*>(p);
}
void reset() {
    for (auto& s : seen) s.clear();
    taken.clear();
    launches = partials_seen = clip_elems = 0;
    place_at = uint64_t(0x1000) << 32;
}
int64_t side() {
    const int64_t kinds[] = {pick(0, 3), pick(1, 64), pick(60, 70), pick(65, 300), pick(1, 700), 64 * pick(1, 20)};
    return kinds[rng() % 6];
}

void run_muon(int count, bool few_large) {
    reset();
    std::vector<zs_muon_matrix> list((size_t)count);
    for (auto& x : list) {
        x.rows = few_large ? pick(3000, 9000) : side();
        x.cols = few_large ? pick(3000, 30000) : side();
        const int64_t n = x.rows * x.cols;
        x.param = fresh(n * 4, 4 * (int)pick(0, 3));
        x.grad = fresh(n * 2, 2 * (int)pick(0, 3));
        x.momentum = static_cast<float*>(fresh(n * 4, 4));
        x.param_bf16 = pick(0, 1) ? static_cast<uint16_t*>(fresh(n * 2, 2)) : nullptr;
        x.scale = 1.0;
    }
    const zs_muon hp = {0.01, 0.9, 0.1, 3.4445, -4.775, 2.0315, 1e-7, 1.0, 0.0, 0.0, 1, (int32_t)pick(1, 6)};
    ws_bytes = muon_step_matrices_workspace_bytes(list.data(), count);
    CHECK(ws_bytes >= 0);
    // group by group, as the launches follow one another: a group's pieces may take the place of the last one's
    int32_t rc = muon_step_matrices(&hp, list.data(), count, ZS_F32, ZS_BF16, nullptr, reinterpret_cast<void*>(kWs), ws_bytes, nullptr);
    CHECK(rc == ZS_OK && partials_seen == 0);
    CHECK(ws_bytes == 0 || muon_step_matrices(&hp, list.data(), count, ZS_F32, ZS_BF16, nullptr, reinterpret_cast<void*>(kWs),
                                              ws_bytes - 1, nullptr) == ZS_EWORKSPACE);
    for (const auto& x : list) {
        const int64_t n = x.rows * x.cols;
        if (n == 0) continue;
        CHECK(seen[1][(uint64_t)(uintptr_t)x.grad] == (n + kMomentumTile - 1) / kMomentumTile);
        CHECK(seen[2][(uint64_t)(uintptr_t)x.grad] == stage_tiles(x.rows, x.cols));
        CHECK(seen[5][(uint64_t)(uintptr_t)x.param] >= 1);
    }
}

template <typename T, typename Need, typename Call>
void run_products(std::vector<T>& list, Need need, Call call) {
    ws_bytes = need(list.data(), (int32_t)list.size());
    CHECK(ws_bytes >= 0 && call(list.data(), (int32_t)list.size(), reinterpret_cast<void*>(kWs), ws_bytes) == ZS_OK);
    for (const auto& x : list) {
        if (seen[0].count((uint64_t)(uintptr_t)x.d) == 0) continue;
        CHECK(seen[0][(uint64_t)(uintptr_t)x.d] >= 1);
    }
}

}  // namespace

int main() {
    for (int count : {0, 1, 2, 7, 119, 241, 1500})
        for (int round = 0; round < (count > 200 ? 2 : 12); ++round) run_muon(count, false);
    // (one group each: pieces of two groups would be told apart by nothing here)
    for (int round = 0; round < 4; ++round) run_muon(2, true);
    for (int dtype : {ZS_F32, ZS_BF16})
        for (int flags = 0; flags < 4; ++flags)
            for (int count : {1, 5, 81, 400}) {
                reset();
                std::vector<zs_product> list((size_t)count);
                int64_t live = 0;
                for (auto& x : list) {
                    x.m = side(), x.n = side(), x.k = side();
                    const int off = pick(0, 1) ? 0 : 4;
                    x.a = fresh(x.m * x.k * 4, off), x.b = fresh(x.k * x.n * 4, off), x.d = fresh(x.m * x.n * 4, 4);
                    x.c = pick(0, 1) ? fresh(x.m * x.n * 4, 4) : nullptr;
                    live += x.m > 0 && x.n > 0;
                }
                run_products(list, [&](const zs_product* p, int32_t n) { return product_add_matrices_workspace_bytes(p, n, dtype, flags); },
                             [&](const zs_product* p, int32_t n, void* ws, int64_t bytes) {
                                 return product_add_matrices(p, n, dtype, ZS_F32, ZS_F32, flags, 1.0, 0.5, ws, bytes, nullptr);
                             });
                CHECK((int64_t)seen[0].size() == live);
                reset();
                std::vector<zs_gram> grams((size_t)count);
                live = 0;
                for (auto& x : grams) {
                    x = zs_gram{};
                    x.rows = side(), x.cols = side(), x.transposed = (int32_t)pick(0, 1);
                    const int64_t s = x.transposed ? x.cols : x.rows;
                    x.a = fresh(x.rows * x.cols * 4, pick(0, 1) ? 0 : 4), x.d = fresh(s * s * 4, 4), x.c = x.d;
                    live += s > 0;
                }
                run_products(grams, [&](const zs_gram* p, int32_t n) { return gram_add_matrices_workspace_bytes(p, n, dtype); },
                             [&](const zs_gram* p, int32_t n, void* ws, int64_t bytes) {
                                 return gram_add_matrices(p, n, dtype, ZS_F32, 1.0, 0.5, ws, bytes, nullptr);
                             });
                CHECK((int64_t)seen[0].size() == live);
            }
    for (int count : {0, 1, 63, 64, 65, 330, 2500})
        for (int round = 0; round < 6; ++round) {
            reset();
            std::vector<zs_mixed_tensor> in((size_t)count), out((size_t)count);
            int64_t parts = 0, elems = 0, empty = 0;
            for (int k = 0; k < count; ++k) {
                const int bits = (int)pick(0, 3);   // both dtypes, said in the addresses too
                const int64_t n = pick(0, 9) == 0 ? 0 : pick(0, 20) == 0 ? pick(1, 1 << 20) : pick(1, 9000);
                in[(size_t)k] = zs_mixed_tensor{fresh(n * 4 + 64, 16 * bits), n, bits & 1 ? ZS_BF16 : ZS_F32, 0};
                out[(size_t)k] = zs_mixed_tensor{fresh(n * 4 + 64, 16 * bits), n, bits & 2 ? ZS_BF16 : ZS_F32, 0};
                parts += (n + mixed_tile_elems(bits & 1) - 1) / mixed_tile_elems(bits & 1);
                elems += n;
                empty += n == 0;
            }
            ws_bytes = grad_norms_sq_tensors_workspace_bytes(in.data(), count);
            double* const result = static_cast<double*>(fresh(8, 0));
            CHECK(grad_norms_sq_tensors(in.data(), count, 1.0, nullptr, result, reinterpret_cast<void*>(kWs), ws_bytes, nullptr) == ZS_OK);
            int64_t got = 0;
            for (const auto& s : seen[6]) got += s.second;
            CHECK(got == parts && partials_seen == 0 && (int64_t)seen[6].size() == count - empty);
            CHECK(grad_clip_tensors(in.data(), out.data(), count, 1.0, 1.0, 0.0, result, nullptr) == ZS_OK && clip_elems == elems);
        }
    std::puts("matrices tables: ok");
    return 0;
}
