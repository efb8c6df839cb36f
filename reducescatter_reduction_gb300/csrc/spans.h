// Overlap among the stretches of memory that a call reads and writes.
#pragma once

#include <algorithm>
#include <cstdio>

#include "comm.h"

namespace ccl {

// A stretch of memory that a call reads or writes.
struct Span {
    Range at;
    const char *name;
    int index;       // rank or tensor; -1: neither
    bool written;
};

constexpr int kMaxSpans = 6 * kMaxRanks + 4;

struct Spans {
    Span s[kMaxSpans];
    int n = 0;
    void add(const char *name, int index, const void *p, uint64_t bytes, bool written)
    {
        if (p && bytes) s[n++] = {{uintptr_t(p), uintptr_t(p) + bytes}, name, index, written};
    }
};

inline ccl_status_t overlap_error(const Span &a, const Span &b)
{
    char at[2][48] = {"", ""};
    const Span *s[2] = {&a, &b};
    for (int i = 0; i < 2; ++i)
        if (s[i]->index >= 0) snprintf(at[i], sizeof at[i], " %d", s[i]->index);
    return fail(CCL_ERR_INVALID_ARG, "%s%s overlaps %s%s", a.name, at[0], b.name, at[1]);
}

// Nothing written overlaps anything else.  Sorts the spans by address: then a
// span meets an earlier one exactly if it begins before the furthest end so
// far (of the written ones, where it is read itself).
inline ccl_status_t check_spans(Span *s, size_t n)
{
    auto before = [](const Span &a, const Span &b) { return a.at.lo < b.at.lo; };
    if (!std::is_sorted(s, s + n, before)) std::sort(s, s + n, before);
    const Span *any = nullptr, *written = nullptr;     // those that reach furthest
    for (size_t i = 0; i < n; ++i) {
        const Span *meets = s[i].written ? any : written;
        if (meets && s[i].at.lo < meets->at.hi) return overlap_error(*meets, s[i]);
        if (!any || s[i].at.hi > any->at.hi) any = &s[i];
        if (s[i].written && (!written || s[i].at.hi > written->at.hi)) written = &s[i];
    }
    return CCL_OK;
}

// A list with a device pointer for each rank.
template <typename P>
inline ccl_status_t check_list(const ccl_comm *c, P const *list, const char *name, size_t align)
{
    if (!list) return fail(CCL_ERR_INVALID_ARG, "%s is NULL", name);
    for (int r = 0; r < c->p; ++r) {
        if (!list[r]) return fail(CCL_ERR_INVALID_ARG, "%s[%d] is NULL", name, r);
        if (uintptr_t(list[r]) % align)
            return fail(CCL_ERR_INVALID_ARG, "%s[%d] is not aligned to its elements (%zu bytes)", name, r, align);
    }
    return CCL_OK;
}

}  // namespace ccl
