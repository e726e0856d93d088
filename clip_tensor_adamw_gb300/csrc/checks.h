// The host-side checks that the operators' entry points share (train_api.cpp, linear_api.cpp, muon_api.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include "host.h"
#include "mica_train.h"

namespace mica {
namespace {

size_t bytes_of(int32_t dtype) { return dtype == MICA_F32 ? 4 : 2; }

bool is_type(int32_t dtype) { return dtype == MICA_F32 || dtype == MICA_F16 || dtype == MICA_BF16; }

// The buffers of one call: each is checked as device memory of the current device, and what is written must not overlap
// anything else. Matrices with the same row stride may interleave (column slices of one buffer).
class Buffers {
  public:
    explicit Buffers(int device) : device_(device) {}

    mica_status vec(const void* p, int64_t count, size_t elem, bool written, const char* name) {
        return span(p, (size_t)count * elem, 0, 0, elem, written, name);
    }

    // rows x cols with the row stride ld; nothing when it is empty
    mica_status matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem, size_t align, bool written,
                       const char* name) {
        if (rows == 0 || cols == 0) return MICA_OK;
        return span(p, ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * elem, (size_t)ld * elem, (size_t)cols * elem,
                    align, written, name);
    }

    // the written buffer at `p` is also read, element by element in place
    void in_place(const void* p) { alias_ = reinterpret_cast<uintptr_t>(p); }

    mica_status disjoint() const {
        for (int i = 0; i < count_; ++i)
            for (int j = 0; j < count_; ++j) {
                const Span &a = list_[i], &b = list_[j];
                if (i == j || !a.written || (b.written && j < i) || a.lo >= b.hi || b.lo >= a.hi) continue;
                if (alias_ && a.lo == alias_ && b.lo == alias_ && a.hi == b.hi && !b.written) continue;
                if (a.stride && a.stride == b.stride) {  // where b's columns fall in a's rows
                    const size_t d = b.lo >= a.lo ? (b.lo - a.lo) % a.stride
                                                  : (a.stride - (a.lo - b.lo) % a.stride) % a.stride;
                    if (d >= a.width && d + b.width <= a.stride) continue;
                }
                return fail(MICA_ERR_OVERLAP, "%s overlaps %s", a.name, b.name);
            }
        return MICA_OK;
    }

  private:
    static constexpr int kMost = 12;  // more than any call's buffers
    struct Span {
        uintptr_t lo, hi;
        size_t stride, width;  // bytes; 0 for a vector
        bool written;
        const char* name;
    };

    mica_status span(const void* p, size_t bytes, size_t stride, size_t width, size_t align, bool written,
                     const char* name) {
        if (bytes == 0) return MICA_OK;
        if (!p) return fail(MICA_ERR_NULL, "%s is NULL", name);
        if (count_ == kMost) return fail(MICA_ERR_COUNT, "%s: too many buffers", name);
        const mica_status s = check_device_span(p, bytes, align, device_, name, 0);
        if (s != MICA_OK) return s;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        list_[count_++] = Span{lo, lo + bytes, stride, width, written, name};
        return MICA_OK;
    }

    int device_;
    uintptr_t alias_ = 0;
    int count_ = 0;
    Span list_[kMost];
};

#define MICA_TRY(x)                            \
    do {                                       \
        const mica_status try_s = (x);         \
        if (try_s != MICA_OK) return try_s;    \
    } while (0)

mica_status check_extent(int64_t rows, int64_t cols, int64_t least_cols, const char* what) {
    if (rows < 0 || rows > MICA_MAX_ROWS)
        return fail(MICA_ERR_COUNT, "%s: %lld rows are outside [0, 2^30]", what, (long long)rows);
    if (cols < least_cols || cols > MICA_MAX_COLS)
        return fail(MICA_ERR_COUNT, "%s: %lld columns are outside [%lld, 2^24]", what, (long long)cols,
                    (long long)least_cols);
    return MICA_OK;
}

// A row stride, and with it the span of `rows` x `cols` elements (both checked), which no larger than 2^44 (16 TB of bytes)
// can be multiplied by an element's size, and added to an address, without wrapping round.
mica_status check_stride(int64_t ld, int64_t least, int64_t rows, int64_t cols, const char* what) {
    if (ld < least || ld > ((int64_t)1 << 40))
        return fail(MICA_ERR_COUNT, "%s: the row stride %lld is outside [%lld, 2^40]", what, (long long)ld,
                    (long long)least);
    if (rows > 1 && ld > (((int64_t)1 << 44) - cols) / (rows - 1))
        return fail(MICA_ERR_COUNT, "%s: %lld rows with the stride %lld span more than 2^44 elements", what,
                    (long long)rows, (long long)ld);
    return MICA_OK;
}

}  // namespace
}  // namespace mica
