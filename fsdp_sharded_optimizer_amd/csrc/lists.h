// Host side of the calls over lists: overlap checks, and tables of launches
// filled entry by entry (internal).
#pragma once

#include <algorithm>
#include <cstdlib>
#include <cstring>

#include "api_common.h"
#include "tensors.h"

namespace zs {
namespace {

// The byte ranges of one call, and whether any written one shares a byte with
// another.  Merged in address order: a list of some hundred tensors has
// thousands of buffers (pairwise: milliseconds).  They come tensor after
// tensor, one kind of buffer at a time in ascending order for most programs
// (views of one buffer, an allocator that moves up), so each kind is kept as a
// sequence of its own, sorted only if it is not in order, and the sequences
// are walked together.
struct Range {
    uintptr_t lo, hi;
};

class Ranges {
public:
    static constexpr int kKinds = 5;
    // room for `count` ranges of each kind; false: no memory
    bool reserve(int32_t count, int kinds) {
        per_ = (int64_t)count;
        const int64_t most = per_ * kinds;
        all_ = most <= kFew ? few_ : static_cast<Range*>(std::malloc((size_t)most * sizeof(Range)));
        return all_ != nullptr;
    }
    Ranges() = default;
    Ranges(const Ranges&) = delete;
    Ranges& operator=(const Ranges&) = delete;
    ~Ranges() {
        if (all_ != few_) std::free(all_);
    }
    void add(int kind, const void* p, int64_t bytes, bool written) {
        if (p == nullptr || bytes <= 0) return;
        Range* const r = all_ + kind * per_;
        int64_t& n = count_[kind];
        written_[kind] = written;
        r[n] = Range{addr(p), addr(p) + (uintptr_t)bytes};
        if (n > 0 && r[n].lo < r[n - 1].lo) sorted_[kind] = false;
        ++n;
    }
    // one range more that is read (the norm, the scalars)
    void add_read(const void* p, int64_t bytes) {
        if (p != nullptr) extra_[extras_++] = Range{addr(p), addr(p) + (uintptr_t)bytes};
    }
    bool clash() {
        int64_t at[kKinds] = {};
        for (int k = 0; k < kKinds; ++k)
            if (!sorted_[k])
                std::sort(all_ + k * per_, all_ + k * per_ + count_[k],
                          [](const Range& a, const Range& b) { return a.lo < b.lo; });
        uintptr_t written_to = 0, any_to = 0;   // how far the ranges before this one reach
        for (;;) {
            int next = -1;
            uintptr_t lo = 0;
            for (int k = 0; k < kKinds; ++k) {
                if (at[k] == count_[k]) continue;
                const uintptr_t x = all_[k * per_ + at[k]].lo;
                if (next < 0 || x < lo) next = k, lo = x;
            }
            if (next < 0) break;
            const Range& r = all_[next * per_ + at[next]++];
            if (r.lo < written_to || (written_[next] && r.lo < any_to)) return true;
            any_to = std::max(any_to, r.hi);
            if (!written_[next]) continue;
            written_to = std::max(written_to, r.hi);
            for (int x = 0; x < extras_; ++x)
                if (r.lo < extra_[x].hi && extra_[x].lo < r.hi) return true;
        }
        return false;
    }

private:
    static constexpr int64_t kFew = 512;
    Range few_[kFew];
    Range* all_ = few_;
    int64_t per_ = 0;
    int64_t count_[kKinds] = {};
    bool written_[kKinds] = {};
    bool sorted_[kKinds] = {true, true, true, true, true};
    Range extra_[2];
    int extras_ = 0;
};

// The sum of the list's numels, or -1 for a bad list.
template <typename T>
int64_t list_total(const T* list, int32_t count) {
    if (count < 0 || (count > 0 && list == nullptr)) return -1;
    int64_t total = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (!size_ok(list[k].numel) || total > kMaxElems - list[k].numel) return -1;
        total += list[k].numel;
    }
    return total;
}

// Fills launches with entries: `launch(batch, tiles)` for each full table.
template <typename Batch, typename Launch>
class Filler {
public:
    Filler(Batch& b, Launch launch) : b_(b), launch_(launch) { clear(); }
    // room for an entry of `tiles` workgroups; the entry's place in out
    int32_t add(int64_t tiles, int& out) {
        if (count_ == Table::kMax || tiles_ + tiles > kListMaxTiles) {
            const int32_t rc = flush();
            if (rc != ZS_OK) return rc;
        }
        out = count_;
        b_.tab.start[count_++] = (uint32_t)tiles_;
        tiles_ += tiles;
        return ZS_OK;
    }
    int32_t flush() {
        if (tiles_ == 0) {   // nothing but tensors without elements
            clear();
            return ZS_OK;
        }
        auto& tab = b_.tab;
        tab.start[count_] = (uint32_t)tiles_;
        tab.shift = 0;
        while (((tiles_ - 1) >> tab.shift) >= kListBuckets) ++tab.shift;
        constexpr int kPer = Table::kPerWord;
        std::memset(tab.bucket, 0, sizeof(tab.bucket));
        int t = 0;
        for (int part = 0; part < kListBuckets && ((int64_t)part << tab.shift) < tiles_; ++part) {
            while ((int64_t)tab.start[t + 1] <= ((int64_t)part << tab.shift)) ++t;
            tab.bucket[part / kPer] |= (uint32_t)t << (Table::kBits * (part % kPer));
        }
        const int32_t rc = hip_status(launch_(b_, tiles_));
        clear();
        return rc;
    }

private:
    using Table = decltype(Batch::tab);
    void clear() {
        for (uint32_t& s : b_.tab.start) s = kNoTile;
        count_ = 0;
        tiles_ = 0;
    }
    Batch& b_;
    Launch launch_;
    int count_ = 0;
    int64_t tiles_ = 0;
};

// Scalars as the kernels hold them, in binary32
inline bool finite_float(double x) { return std::isfinite((float)x); }
inline bool positive_float(double x) { return (float)x > 0.0f && finite_float(x); }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T>
T* advance(T* p, int64_t bytes) {
    return p == nullptr ? nullptr : reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes);
}

}  // namespace
}  // namespace zs
