// The sums that a step's pages follow from, and whether it can be carried out
// (assign_kernels.hip runs this; it runs on the host as well).
#pragma once

#include <climits>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "token_internal.h"

namespace bevpool {

struct AssignSums { uint32_t tokens, taken, returned; };

// Tokens may pass 32 bits before the step is refused for it: they stop at 2^32 - 1,
// which is past any room there can be.  Pages are at most a table's entries.
__host__ __device__ __forceinline__ AssignSums operator+(AssignSums a, AssignSums b)
{
    return {__builtin_elementwise_add_sat(a.tokens, b.tokens), a.taken + b.taken, a.returned + b.returned};
}

struct AssignLengths { int keep, fresh, before, after; bool fits; };

// A sequence's three lengths as they are given.
struct AssignGiven { int kv, keep, fresh; };

__host__ __device__ __forceinline__ AssignLengths lengths_of(const AssignParams &p, const AssignGiven &g)
{
    const int64_t room = int64_t(p.max_pages) << p.page_shift;
    const int page = (1 << p.page_shift) - 1;
    AssignLengths l;
    l.fits = g.kv <= room;
    const int kv = g.kv < 0 ? 0 : (l.fits ? g.kv : int(room));
    l.keep = g.keep < 0 ? 0 : (g.keep > kv ? kv : g.keep);
    l.fresh = g.fresh > 0 ? g.fresh : 0;
    l.fits = l.fits && l.keep + int64_t(l.fresh) <= room;
    if (!l.fits) l.fresh = 0;                          // the step is refused
    l.before = int((kv + int64_t(page)) >> p.page_shift);
    l.after = int((l.keep + int64_t(l.fresh) + page) >> p.page_shift);
    return l;
}

__host__ __device__ __forceinline__ AssignSums sums_of(const AssignLengths &l)
{
    const int more = l.after - l.before;
    return {uint32_t(l.fresh), uint32_t(more > 0 ? more : 0), uint32_t(more < 0 ? -more : 0)};
}

// The step of these sums over all sequences, with `listed` pages said to be free.
// After it, left are (if it is not refused).
__host__ __device__ __forceinline__ AssignStep step_of(const AssignParams &p, const AssignSums &all, bool fits,
                                                       int listed, int64_t &left)
{
    const int count = listed < 0 ? 0 : (listed > p.n_free ? p.n_free : listed);
    // the list has room for what comes back
    left = int64_t(count) + all.returned - all.taken;
    const int status = !fits || all.tokens > uint32_t(p.n_tokens) || left > p.n_free ? -1
                       : (left < 0 ? int(-left) : 0);
    return {status, status ? 0 : int(all.taken), status ? 0 : int(all.returned), count};
}

}  // namespace bevpool
