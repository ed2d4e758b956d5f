// The tables that the calls over lists of tensors launch with, replayed on the
// host under AddressSanitizer and UndefinedBehaviorSanitizer: the entry points'
// source with launches that look a table up as the kernels do, for every
// workgroup, and check which elements of which tensor it would take and where
// (run by tests/test_tensors_tables.py).  Addresses are made up and never used.
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

constexpr uint64_t kWindow = uint64_t(1) << 40;

template <int N>
uint32_t find(const ListTable<N>& tab, uint32_t w) {
    using Table = ListTable<N>;
    const uint32_t part = w >> tab.shift;
    CHECK(part < (uint32_t)kListBuckets);
    uint32_t t = tab.bucket[part / Table::kPerWord] >> (Table::kBits * (part % Table::kPerWord)), from;
    t &= (1u << Table::kBits) - 1;
    do {
        from = t;
        CHECK(from < (uint32_t)N);
        for (int k = 1; k <= kListScan; ++k) t += w >= tab.start[from + k] ? 1 : 0;
    } while (t == from + kListScan);
    CHECK(t < (uint32_t)N && tab.start[t] <= w && w < tab.start[t + 1]);
    return t;
}

// one tensor of the list under test and how far workgroups have covered it
struct Tensor {
    uint64_t ptr[5];   // 0: none
    int64_t numel, done;
};
std::vector<Tensor> list;
int64_t size_of[5];   // bytes per element of each stream
int launches;
int64_t norm_total;

void start() {
    for (Tensor& t : list) t.done = 0;
    launches = 0;
    norm_total = 0;
}
void all_done() {
    for (const Tensor& t : list) CHECK(t.done == t.numel);
}

uint64_t addr40(const Q8Batch& b, uint32_t t, int j) {
    return (uint64_t)b.e[t].lo[j] | (uint64_t)(b.e[t].hi >> (8 * j) & 0xFFu) << 32 |
           (uint64_t)(b.top >> (8 * j) & 0xFFu) << 40;
}

hipError_t q8_launch(const Q8Batch& b, int64_t tiles) {
    ++launches;
    for (int64_t w = 0; w < tiles; ++w) {
        const uint32_t t = find(b.tab, (uint32_t)w), first = b.tab.start[t], next = b.tab.start[t + 1];
        const uint32_t tail = b.tail[t / 2] >> (16 * (t % 2));
        const int64_t n = w + 1 == next ? (int64_t)(tail & kQ8Tail) + 1 : kQ8Pad;
        const int64_t entry = (w - first) * kQ8Pad, off = (int64_t)b.off * kLaunchElems;
        CHECK(b.index + t < list.size());
        Tensor& x = list[b.index + t];
        CHECK(x.done == off + entry && x.done + n <= x.numel);
        x.done += n;
        const uint32_t has[4] = {kQ8Has0, kQ8Has1, 0, kQ8Has3};
        for (int j = 0; j < 4; ++j) {
            if (j != 2) CHECK(((tail & has[j]) != 0) == (x.ptr[j] != 0));
            if (j != 2 && x.ptr[j] != 0)
                CHECK(addr40(b, t, j) + (uint64_t)(entry * size_of[j]) == x.ptr[j] + (uint64_t)((off + entry) * size_of[j]));
        }
        CHECK(addr40(b, t, 2) == x.ptr[2]);
        const int64_t padded = (b.padded != 0 ? (int64_t)b.padded : (int64_t)(next - first)) * kQ8Pad;
        CHECK(padded == q8_padded(x.numel));
    }
    return hipSuccess;
}

}  // namespace

namespace zs {

int64_t norm_tile_elems(int bf16) { return bf16 ? 8192 : 4096; }
hipError_t launch_norm_tensors(const NormBatch& b, int bf16, bool, int64_t tiles, float, double*, hipStream_t) {
    ++launches;
    static size_t at = 0;   // the tensor that the last workgroup was in
    if (norm_total == 0) at = 0;
    const int64_t tile = norm_tile_elems(bf16);
    for (int64_t w = 0; w < tiles; ++w) {
        const uint32_t t = find(b.tab, (uint32_t)w);
        const int64_t entry = (w - b.tab.start[t]) * tile;
        const int64_t n = w + 1 == b.tab.start[t + 1] ? (int64_t)(b.e[t].hi_tail >> 16) + 1 : tile;
        while (list[at].done == list[at].numel) ++at;
        Tensor& x = list[at];
        const uint64_t p = (uint64_t)b.e[t].lo | (uint64_t)(b.e[t].hi_tail & 0xFFFFu) << 32;
        CHECK(p + (uint64_t)(entry * size_of[0]) == x.ptr[0] + (uint64_t)(x.done * size_of[0]) && x.done + n <= x.numel);
        x.done += n;
        norm_total += n;
    }
    return hipSuccess;
}
hipError_t launch_list_sum(const double*, int64_t, double*, double*, hipStream_t) { return hipSuccess; }
hipError_t launch_adamw_tensors(const AdamwBatch& b, int, int, bool, bool, int64_t tiles, hipStream_t) {
    ++launches;
    static size_t at = 0;
    if (launches == 1) at = 0;
    for (int64_t w = 0; w < tiles; ++w) {
        const uint32_t t = find(b.tab, (uint32_t)w);
        const AdamwEntry& e = b.e[t];
        uint64_t p[5];
        for (int j = 0; j < 5; ++j)
            p[j] = (uint64_t)e.lo[j] | (uint64_t)(e.hi[j / 2] >> (16 * (j % 2)) & 0xFFFFu) << 32;
        int64_t lo = (w - b.tab.start[t]) * kListTile - (e.hi[2] >> 16), hi = lo + kListTile;
        lo = lo < 0 ? 0 : lo, hi = hi > (int64_t)e.numel ? (int64_t)e.numel : hi;
        while (lo < hi) {   // a tile may run on into neighbours that follow one another
            while (list[at].done == list[at].numel) ++at;
            Tensor& x = list[at];
            const int64_t n = hi - lo < x.numel - x.done ? hi - lo : x.numel - x.done;
            for (int j = 0; j < 5; ++j) {
                if (x.ptr[j] == 0) CHECK(p[j] == 0);
                else CHECK(p[j] + (uint64_t)(lo * size_of[j]) == x.ptr[j] + (uint64_t)(x.done * size_of[j]));
            }
            x.done += n;
            lo += n;
        }
    }
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

uint32_t rng = 12345;
uint32_t draw(uint32_t n) {
    rng = rng * 1664525u + 1013904223u;
    return (rng >> 9) % n;
}

// kind 0: each stream somewhere of its own; 1: all streams back to back; 2: as 0,
// now and then in another window of 1 TiB
void make(int count, int kind, const int64_t* sizes, bool q8, bool copies, bool big) {
    list.clear();
    uint64_t at[5] = {0x700000000000, 0x720000000000, 0x740000000000, 0x760000000000, 0x780000000000};
    for (int j = 0; j < 5; ++j) size_of[j] = sizes[j], at[j] += 256 + 8 * (uint64_t)draw(30);
    if (q8) at[2] = 0x740000000000;
    for (int k = 0; k < count; ++k) {
        Tensor t{};
        const uint32_t what = draw(8);
        t.numel = what == 0 ? 0 : what == 1 ? 1 : what == 2 ? 512 : what == 3 ? 256 + draw(3) : 1 + draw(20000);
        if (big && k == count / 2) t.numel = kLaunchElems + 70001;
        const bool copy = copies && (kind == 1 || draw(3) != 0);
        for (int j = 0; j < 5; ++j) {
            if (kind != 1) at[j] += 16 * (uint64_t)draw(1000) + (draw(2) ? (uint64_t)size_of[j] * draw(8) : 0);
            if (kind == 2 && draw(20) == 0) at[j] = (at[j] ^ kWindow) + (uint64_t(1) << 33);
            if (q8 && j == 2) at[j] = (at[j] + 15) / 16 * 16;
            t.ptr[j] = at[j];
            at[j] += q8 && j == 2 ? (uint64_t)moments_q8_bytes(t.numel) : (uint64_t)(t.numel * size_of[j]);
        }
        if (!copy) t.ptr[q8 ? 3 : 4] = 0;
        if (q8) t.ptr[4] = 0;
        list.push_back(t);
    }
}

template <typename T>
T* as(uint64_t p) { return reinterpret_cast<T*>((uintptr_t)p); }

void steps(int count, int kind, bool big) {
    zs_adamw hp{};
    hp.step = 1, hp.lr = 1e-3, hp.beta1 = 0.9, hp.beta2 = 0.95, hp.eps = 1e-8, hp.grad_scale = 1.0;
    for (int bf16 = 0; bf16 < 2; ++bf16) {
        const int64_t psz = bf16 ? 2 : 4, gsz = bf16 ? 4 : 2;
        const int32_t pd = bf16 ? ZS_BF16 : ZS_F32, gd = bf16 ? ZS_F32 : ZS_BF16;
        {
            const int64_t sizes[5] = {psz, gsz, 4, 4, 2};
            make(count, kind, sizes, false, !bf16, big);
            std::vector<zs_adamw_tensor> c;
            for (const Tensor& t : list)
                c.push_back({as<void>(t.ptr[0]), as<const void>(t.ptr[1]), as<float>(t.ptr[2]), as<float>(t.ptr[3]),
                             as<uint16_t>(t.ptr[4]), t.numel});
            start();
            CHECK(adamw_step_tensors(&hp, c.data(), count, pd, gd, nullptr, nullptr) == ZS_OK);
            all_done();
            if (kind == 1 && !big) CHECK(launches <= 1);
            if (kind == 0 && !big) CHECK(launches <= (count + 97) / 98);
        }
        {
            const int64_t sizes[5] = {psz, gsz, 1, 2, 1};
            make(count, kind, sizes, true, !bf16, big);
            std::vector<zs_adamw_q8_tensor> c;
            for (const Tensor& t : list)
                c.push_back({as<void>(t.ptr[0]), as<const void>(t.ptr[1]), as<void>(t.ptr[2]), as<uint16_t>(t.ptr[3]), t.numel});
            start();
            CHECK(adamw_step_tensors_q8(&hp, 7, c.data(), count, pd, gd, nullptr, nullptr) == ZS_OK);
            all_done();
            if (kind != 2 && !big) CHECK(launches <= (count + 149) / 150);
        }
        {
            const int64_t sizes[5] = {psz, psz, 1, 1, 1};
            make(count, kind, sizes, true, false, big);
            std::vector<zs_moments_q8> c;
            for (Tensor& t : list) {
                if (draw(4) == 0) t.ptr[draw(2)] = 0;
                c.push_back({as<void>(t.ptr[0]), as<void>(t.ptr[1]), as<void>(t.ptr[2]), t.numel});
            }
            start();
            CHECK(moments_q8_encode(c.data(), count, pd, 3, nullptr) == ZS_OK);
            all_done();
            for (size_t k = 0; k < list.size(); ++k)
                if (draw(5) == 0) {   // nothing to read out of these
                    c[k].exp_avg = c[k].exp_avg_sq = nullptr;
                    list[k].ptr[0] = list[k].ptr[1] = 0;
                }
            start();
            CHECK(moments_q8_decode(c.data(), count, pd, nullptr) == ZS_OK);
            for (const Tensor& t : list) CHECK(t.done == (t.ptr[0] == 0 && t.ptr[1] == 0 ? 0 : t.numel));
        }
        {
            const int64_t sizes[5] = {gsz, 1, 1, 1, 1};
            make(count, kind, sizes, false, false, big);
            std::vector<zs_tensor> c(list.size());
            for (size_t k = 0; k < list.size(); ++k) c[k].ptr = as<void>(list[k].ptr[0]), c[k].numel = list[k].numel;
            const int64_t need = grad_norm_sq_tensors_workspace_bytes(c.data(), count, gd);
            start();
            CHECK(grad_norm_sq_tensors(c.data(), count, gd, 1.0, as<double>(0x100000), as<void>(0x200000), need, nullptr) ==
                  ZS_OK);
            all_done();
            if (!big) CHECK(launches <= (count + 327) / 328);
        }
    }
}

}  // namespace

int main() {
    for (int count : {0, 1, 2, 97, 98, 99, 149, 150, 151, 152, 255, 256, 257, 327, 328, 329, 700})
        for (int kind = 0; kind < 3; ++kind)
            for (int again = 0; again < 3; ++again) steps(count, kind, false);
    for (int count : {1, 3, 160})
        for (int kind = 0; kind < 3; ++kind) steps(count, kind, true);
    std::printf("tables: ok\n");
    return 0;
}
