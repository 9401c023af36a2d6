// Block tables, offsets and slot maps from request lengths (gfx950).  See bevpool.h
// for the definition.
//
// Three running sums over the sequences decide everything: their new tokens, the
// pages each takes and the pages each gives back.  One block of threads makes
// them (a wave has consecutive sequences, the waves' sums meet in LDS), and with
// the totals at hand either carries the step out or refuses it.  What is left has
// no order: a wave finds the sequences of 64 tokens, and a token its page in the
// table or, where the page is a new one, at the place in the free list that the
// page's number names; so does a table entry.  No thread waits for what another
// writes: entries that are given back are read and stay, entries that are taken are
// written and not read, and the free list is read below its old end or written
// above it, never both.
//
// Bound by latency.  Small steps are one launch: the block that makes the sums
// goes on to the tokens (64 requests of a token 4.4 us).  For larger ones a second
// launch has a thread for each: 4096 requests of up to five tokens 6.3 + 5.9 us, 96
// prompts of up to 8191 tokens 3.1 + 5.3.
#include <hip/hip_runtime.h>

#include "assign_plan.h"
#include "token_device.h"

namespace bevpool {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kLanes;
constexpr int kSpreadThreads = 256, kSpreadBlocks = 2048;
// Tokens, and pages taken for them, that one block deals with.  Pages that are given
// back are not among them: only the lengths on the device tell how many there are.  In
// a step of few tokens they go by the one block: 64 requests that end with 512 pages
// each take 41 us, with 7500 each (480,000 pages) 535, one of them with 7500 12.
constexpr int kWholeItems = 4096;

using Seq = AssignSeq;
using Step = AssignStep;

using Sums = AssignSums;
using Lengths = AssignLengths;
using Given = AssignGiven;

// Another lane's, by a shift or broadcast within the vector pipe; 0 where CTRL names
// none, or where ROWS leaves the lane out.
template <int CTRL, int ROWS>
__device__ __forceinline__ Sums moved(Sums a)
{
    const auto of = [](uint32_t x) { return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, ROWS, 0xf, false)); };
    return {of(a.tokens), of(a.taken), of(a.returned)};
}

// Of the lanes up to this one, by the whole wave; and of all of them.
__device__ __forceinline__ Sums upto_lane(Sums a)
{
    a = moved<0x111, 0xf>(a) + a;          // rows of 16: from 1, 2, 4 and 8 lanes below
    a = moved<0x112, 0xf>(a) + a;
    a = moved<0x114, 0xf>(a) + a;
    a = moved<0x118, 0xf>(a) + a;
    a = moved<0x142, 0xa>(a) + a;          // lane 15 of rows 0 and 2 to the rows after them
    return moved<0x143, 0xc>(a) + a;       // lane 31 to the upper half
}

__device__ __forceinline__ Sums last_lane(Sums a)
{
    const auto of = [](uint32_t x) { return uint32_t(__builtin_amdgcn_readlane(int(x), kLanes - 1)); };
    return {of(a.tokens), of(a.taken), of(a.returned)};
}

__device__ __forceinline__ Given given_of(const AssignParams &p, int s)
{
    return {p.kv_lengths[s], p.keep_lengths ? p.keep_lengths[s] : INT32_MAX, p.new_lengths[s]};
}

// The last of n non-decreasing values key(i) that is at most x, from key(0) <= x.
template <typename Key>
__device__ __forceinline__ int last_upto(int n, int x, Key key)
{
    int lo = 0, len = n;
    while (len > 1) {
        const int half = len / 2;
        if (key(lo + half) <= x) {
            lo += half;
            len -= half;
        } else {
            len = half;
        }
    }
    return lo;
}

// The r-th page given back: an entry of its sequence's row past what it keeps.
__device__ __forceinline__ int returned_page(const AssignParams &p, const Seq *seqs, int r)
{
    const int s = last_upto(p.n_seqs, r, [&](int i) { return seqs[i].returned; });
    // its pages end at before, those that it gives back with the next one's first
    const int next = s + 1 < p.n_seqs ? seqs[s + 1].returned : p.step->returned;
    const int first = seqs[s].before - (next - seqs[s].returned);
    return p.block_table[int64_t(s) * p.max_pages + first + r - seqs[s].returned];
}

__device__ __forceinline__ int taken_page(const AssignParams &p, const Seq *seqs, const Step &step, int i)
{
    if (i < step.returned) return returned_page(p, seqs, i);
    return p.free_pages[step.count - 1 - (i - step.returned)];
}

// The owner of each lane's item, which are 64 consecutive ones from n on (the wave's;
// none past the last): the last sequence whose key is at most it.  One search by the
// wave for the first of them, then the next 64 keys lie in lanes and are searched
// there; where more than 64 sequences begin among them, each lane searches by itself.
template <typename Key>
__device__ __forceinline__ int owner(int n_seqs, int n, Key key)
{
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int first = count_upto(n_seqs - 1, n, key);
    const int at = first + 1 + lane;
    const int next = at < n_seqs ? key(at) : INT32_MAX;
    const int mine = n + lane;
    if (__shfl(next, kLanes - 1) <= n + kLanes - 1) return last_upto(n_seqs, mine, key);
    int lo = 0;                                 // of the keys in lanes, how many are at most it
#pragma unroll
    for (int step = kLanes / 2; step > 0; step /= 2)
        if (__shfl(next, lo + step - 1) <= mine) lo += step;
    return first + lo;
}

// Items in the waves' turns: tokens, then table entries, then pages that go back to
// the list, each kind from a multiple of 64 on.
__device__ __forceinline__ void carry_out(const AssignParams &p, const Seq *seqs, const Step &step, int wave, int waves)
{
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int tokens = p.q_offsets[p.n_seqs], back = max(step.returned - step.taken, 0);
    const auto turns = [](int n) { return (int64_t(n) + kLanes - 1) / kLanes; };
    const int64_t to_tokens = turns(p.n_tokens), to_entries = to_tokens + turns(step.taken);
    const int64_t end = to_entries + turns(back);
    for (int64_t turn = wave; turn < end; turn += waves) {
        if (turn < to_tokens) {
            const int base = int(turn) * kLanes;
            int slot = -1, place = -1;
            if (base < tokens) {
                const int s = owner(p.n_seqs, base, [&](int i) { return p.q_offsets[i]; });
                if (base + lane < tokens) {
                    const Seq q = seqs[s];
                    place = q.keep + base + lane - p.q_offsets[s];
                    const int entry = place >> p.page_shift;
                    const int page = entry < q.before ? p.block_table[int64_t(s) * p.max_pages + entry]
                                                      : taken_page(p, seqs, step, q.taken + entry - q.before);
                    if (page >= 0 && page < p.n_pages)
                        slot = (page << p.page_shift) + (place & ((1 << p.page_shift) - 1));
                }
            }
            if (base + lane < p.n_tokens) {
                if (p.slots) p.slots[base + lane] = slot;
                if (p.places) p.places[base + lane] = place;
            }
        } else if (turn < to_entries) {
            const int base = int(turn - to_tokens) * kLanes;
            const int s = owner(p.n_seqs, base, [&](int i) { return seqs[i].taken; });
            const int i = base + lane;
            if (i < step.taken)
                p.block_table[int64_t(s) * p.max_pages + seqs[s].before + i - seqs[s].taken] =
                    taken_page(p, seqs, step, i);
        } else {
            const int64_t r = (turn - to_entries) * kLanes + lane + step.taken;
            if (r < step.returned)
                p.free_pages[int64_t(step.count) + step.returned - 1 - r] = returned_page(p, seqs, int(r));
        }
    }
}

// One block.  Whole: it carries the step out as well.
template <bool WHOLE>
__global__ __launch_bounds__(kThreads) void plan_step(AssignParams p)
{
    __shared__ Sums wave_sums[kWaves];
    __shared__ int bad, listed;
    const int tid = int(threadIdx.x), lane = tid & (kLanes - 1), wave = tid / kLanes;
    // a wave's sequences follow each other, 64 at a time side by side in its lanes
    const int each = ((p.n_seqs + kThreads - 1) / kThreads) * kLanes;
    const int first = min(wave * each, p.n_seqs), last = min(first + each, p.n_seqs);
    const auto given = [&](int s) { return s < last ? given_of(p, s) : Given{0, 0, 0}; };
    if (tid == 0) {
        bad = 0;
        listed = *p.free_count;          // next_free may be the same
    }
    __syncthreads();

    // the first four 64s stay in registers; there are no more up to 4096 sequences
    constexpr int kKept = 4;
    Given kept[kKept];
    Sums upto[kKept], own = {0, 0, 0};
    bool fits = true;
#pragma unroll
    for (int i = 0; i < kKept; ++i) kept[i] = i * kLanes < each ? given(first + i * kLanes + lane) : Given{0, 0, 0};
    for (int s = first + kKept * kLanes + lane; s < first + each; s += kLanes) {
        const Lengths l = lengths_of(p, given(s));
        fits &= l.fits;
        own = own + sums_of(l);
    }
    Sums total = each > kKept * kLanes ? last_lane(upto_lane(own)) : own;
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
        if (i * kLanes >= each) continue;
        const Lengths l = lengths_of(p, kept[i]);
        fits &= l.fits;
        upto[i] = upto_lane(sums_of(l));
        total = total + last_lane(upto[i]);
    }
    if (!fits) bad = 1;
    if (lane == 0) wave_sums[wave] = total;
    __syncthreads();
    Sums all = {0, 0, 0}, at = {0, 0, 0};
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) at = all;
        all = all + wave_sums[w];
    }
    int64_t left;
    const Step step = step_of(p, all, !bad, listed, left);
    const int status = step.refused;
    const auto write = [&](int s, const Given &g, Sums with) {
        const Lengths l = lengths_of(p, g);
        const Sums own = sums_of(l);       // of a step that is not refused no sum has stopped
        const Sums mine = at + Sums{with.tokens - own.tokens, with.taken - own.taken, with.returned - own.returned};
        if (s < last) {
            p.q_offsets[s] = status ? 0 : int(mine.tokens);
            p.seqs[s] = {l.keep, l.before, int(mine.taken), int(mine.returned)};
            p.next_lengths[s] = status ? g.kv : l.keep + l.fresh;      // may be kv_lengths
        }
        at = at + last_lane(with);
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (i * kLanes < each) write(first + i * kLanes + lane, kept[i], upto[i]);
    for (int s = first + kKept * kLanes + lane; s < first + each; s += kLanes) {
        const Given g = given(s);
        write(s, g, upto_lane(sums_of(lengths_of(p, g))));
    }
    if (tid == 0) {
        p.q_offsets[p.n_seqs] = status ? 0 : int(all.tokens);
        *p.step = step;
        *p.status = status;
        *p.next_free = status ? listed : int(left);
    }
    if constexpr (WHOLE) {
        __syncthreads();
        carry_out(p, p.seqs, step, wave, kWaves);
    }
}

__global__ __launch_bounds__(kSpreadThreads) void spread_step(AssignParams p)
{
    constexpr int kHere = kSpreadThreads / kLanes;
    carry_out(p, p.seqs, *p.step, int(blockIdx.x) * kHere + int(threadIdx.x) / kLanes, int(gridDim.x) * kHere);
}

}  // namespace

size_t assign_workspace_bytes(int32_t n_seqs)
{
    return 256 + ((size_t(n_seqs) * sizeof(Seq) + 255) & ~size_t(255));
}

hipError_t run_assign_pages(AssignParams &p, void *workspace, hipStream_t stream)
{
    p.step = static_cast<Step *>(workspace);
    p.seqs = reinterpret_cast<Seq *>(static_cast<char *>(workspace) + 256);
    // a sequence takes at most new / page_size + 1 pages
    const int64_t items = int64_t(p.n_tokens) + (p.n_tokens >> p.page_shift) + p.n_seqs + 2 * kLanes;
    if (items <= kWholeItems) {
        plan_step<true><<<1, kThreads, 0, stream>>>(p);
        return hipGetLastError();
    }
    plan_step<false><<<1, kThreads, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = (items + kSpreadThreads - 1) / kSpreadThreads;
    spread_step<<<uint32_t(blocks < kSpreadBlocks ? blocks : kSpreadBlocks), kSpreadThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace bevpool
