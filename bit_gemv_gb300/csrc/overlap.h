// Whether two tensors of a call share memory, exactly: views of one buffer that lie between each other's rows do not.
#pragma once

#include <algorithm>
#include <cstdint>

namespace ninfer {

// `run` bytes at base + i * stride[0] + j * stride[1] for i < count[0], j < count[1], the outer dimension first.
struct Span {
    uint64_t at = 0, run = 0, count[2] = {1, 1}, stride[2] = {0, 0};

    Span() = default;
    Span(const void *p, uint64_t bytes) : at(reinterpret_cast<uint64_t>(p)), run(p ? bytes : 0) {}
    Span(const void *p, uint64_t bytes, uint64_t rows, uint64_t row_stride, uint64_t parts = 1, uint64_t part_stride = 0) : Span(p, bytes) {
        count[0] = rows, stride[0] = row_stride;
        count[1] = parts, stride[1] = part_stride;
        for (int d = 0; d < 2; ++d)
            if (count[d] <= 1) count[d] = 1, stride[d] = 0;
        if (stride[1] > stride[0]) std::swap(stride[0], stride[1]), std::swap(count[0], count[1]);
        for (int d = 1; d >= 0; --d)        // rows without gaps are one
            if (count[d] > 1 && stride[d] == run && (d == 1 || count[1] == 1)) run *= count[d], count[d] = 1, stride[d] = 0;
        if (count[0] == 1 && count[1] > 1) std::swap(stride[0], stride[1]), std::swap(count[0], count[1]);
    }
    uint64_t end() const { return at + (count[0] - 1) * stride[0] + (count[1] - 1) * stride[1] + run; }
    // The same rows of part j alone.
    Span part(uint64_t j) const {
        Span s = *this;
        s.at += j * stride[1];
        s.count[1] = 1, s.stride[1] = 0;
        return s;
    }
    Span row(uint64_t i) const {
        Span s = *this;
        s.at += i * stride[0];
        s.count[0] = 1, s.stride[0] = 0;
        return s;
    }

    bool meets(const Span &o) const {
        if (!run || !o.run || end() <= o.at || o.end() <= at) return false;
        for (const Span *two : {this, &o})
            if (two->count[1] > 1) {
                const Span &other = two == this ? o : *this;
                for (uint64_t j = 0; j < two->count[1]; ++j)
                    if (two->part(j).meets(other)) return true;
                return false;
            }
        if (count[0] > 1 && o.count[0] > 1 && stride[0] != o.stride[0]) {
            const Span &few = count[0] <= o.count[0] ? *this : o, &many = count[0] <= o.count[0] ? o : *this;
            for (uint64_t i = 0; i < few.count[0]; ++i)
                if (few.row(i).meets(many)) return true;
            return false;
        }
        // rows of one stride S, distance d + k S for k from -(rows - 1) to o's rows - 1: is one of them in (-o.run, run)?
        const __int128 d = (__int128)o.at - at, s = std::max(stride[0], o.stride[0]);
        const __int128 low = -(__int128)(count[0] - 1), high = (__int128)o.count[0] - 1;
        if (!s) return d > -(__int128)o.run && d < (__int128)run;
        const auto floor_div = [](__int128 a, __int128 b) { return a / b - (a % b < 0); };
        const __int128 first = floor_div(-(__int128)o.run - d, s) + 1, last = -floor_div(d - (__int128)run, s) - 1;
        return std::max(first, low) <= std::min(last, high);
    }
    // Whether its rows do not share memory with each other (parts of a row that lie between those of the next count as if they did).
    bool simple() const {
        return (count[1] == 1 || stride[1] >= run) && (count[0] == 1 || stride[0] >= (count[1] - 1) * stride[1] + run);
    }
    bool same(const Span &o) const {
        return at == o.at && run == o.run && std::equal(count, count + 2, o.count) && std::equal(stride, stride + 2, o.stride);
    }
};

}  // namespace ninfer
