// Norm and rotation of query and key heads, its gradient, and the append to a
// paged cache (gfx950).  See bevpool.h for the formulas.
//
// All three are one pass over their rows and bound by HBM where they are
// large: about ten operations for each element read and written.  What decides
// the time is that every load is 16 bytes wide, that a pair's two coordinates
// meet in one lane, and that the angle (fp64 product, reduction, sine and
// cosine: some 60 instructions) is paid once for a token, a pair and a chunk of
// heads.  With few tokens the heads are dealt to more waves, and each works its
// angles out again: 4 times at 16384 tokens of 20 heads, once a head at 4223
// tokens of 10.  So do the append's waves that hold values alone.
//
// Layout.  A row of head_dim elements belongs to LPR lanes (the power of two
// at or above head_dim / 16), each lane holding two runs of eight elements:
// in the halves layout the runs that start at 8j and R/2 + 8j, so both
// coordinates of its eight pairs; in the adjacent layout, and past R, the 16
// elements from 16j.  No coordinate moves between lanes; the mean square is
// the only cross-lane sum.  A wave holds 64 / LPR tokens and walks over heads,
// keeping its eight sines and cosines.
//
// Measured (a 2 GiB copy moves 4.96 TB/s): 16384 tokens of 16 + 4 heads of 128,
// bf16: forward 42 us (4.0 TB/s), backward 54 us (4.7) and 4.6 for the last sum
// of the weight gradient.  Append of 16384 tokens, 16 query heads, 8 key heads
// of 128, bf16 to e4m3: 50 us (4.7 TB/s), of 64 single tokens 6 us: the chain
// offsets, place, page, store.  4223 tokens of 5 + 5 heads of 80, fp32: forward
// 12 us and backward 15 + 4, 2.2 times their bytes: the angles of every head,
// and 3 of 8 lanes without elements.
#include <hip/hip_runtime.h>

#include "token_device.h"

namespace bevpool {
namespace {

constexpr int kBlock = 256;
constexpr int kWavesPerBlock = kBlock / kLanes;

struct Slot {
    int a, b;         // first element of the lane's two runs
    int pair;         // first of its eight pairs, -1 past R
    bool on;          // the lane holds elements
};

__device__ __forceinline__ Slot slot_of(int j, int head_dim, int half, bool adjacent)
{
    Slot s;
    s.on = 16 * j < head_dim;
    const bool turned = 8 * j < half;
    s.pair = turned ? 8 * j : -1;
    s.a = turned && !adjacent ? 8 * j : 16 * j;
    s.b = turned && !adjacent ? half + 8 * j : 16 * j + 8;
    return s;
}

// Cosines and sines of the lane's eight angles.  position * inv_freq has up
// to 55 significant bits and is rounded to fp64's 53; the turn's fraction
// then keeps an absolute error of 2^-53 of the number of turns: two million
// radians out the reduction is right to 2^-30.  Its result is rounded to fp32,
// so at any position the angle that the sine is taken of is right to about
// 2^-23 radians (2^-25 half turns), and no better.
__device__ __forceinline__ void angles(const RopeParams &p, const Slot &s, int token, f32x8 &cs,
                                       f32x8 &sn)
{
    cs = 1.0f;
    sn = 0.0f;
    if (s.pair < 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = s.pair + i;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kMaxRopeAxes - 1; ++a)
            if (a + 1 < p.n_axes && pair >= p.section_end[a]) axis = a + 1;
        const double angle = double(p.positions[int64_t(axis) * p.n_tokens + token]) *
                             double(p.inv_freq[pair]);
        const double turns = angle * 0.15915494309189533577;   // 1 / (2 pi)
        const float half_turns = float(2.0 * (turns - rint(turns)));
        float sv, cv;
        sincospif(half_turns, &sv, &cv);
        cs[i] = cv;
        sn[i] = sv;
    }
}

// Turns the lane's pairs.  A lane past R keeps its elements: a product with
// sine 0 would make NaN of an infinity in its neighbour.
template <bool ADJ>
__device__ __forceinline__ void rotate(f32x8 &a, f32x8 &b, f32x8 cs, f32x8 sn, bool turned)
{
    if (!turned) return;
    if constexpr (ADJ) {
        f32x8 u = __builtin_shufflevector(a, b, 0, 2, 4, 6, 8, 10, 12, 14);
        f32x8 v = __builtin_shufflevector(a, b, 1, 3, 5, 7, 9, 11, 13, 15);
        const f32x8 x = u * cs - v * sn, y = v * cs + u * sn;
        a = __builtin_shufflevector(x, y, 0, 8, 1, 9, 2, 10, 3, 11);
        b = __builtin_shufflevector(x, y, 4, 12, 5, 13, 6, 14, 7, 15);
    } else {
        const f32x8 x = a * cs - b * sn, y = b * cs + a * sn;
        a = x;
        b = y;
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int m = 1; m < LPR; m *= 2) v += __shfl_xor(v, m);
    return v;
}

__device__ __forceinline__ float dot8(f32x8 a, f32x8 b)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
    return s;
}

// Weights of the lane's two runs; all ones without a weight.
template <int DT>
__device__ __forceinline__ void load_weight(const RopeParams &p, const void *w, const Slot &s,
                                            f32x8 &wa, f32x8 &wb)
{
    wa = 1.0f;
    wb = 1.0f;
    if (!w || !s.on) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (p.weight_dtype == kF32) {
            wa[i] = static_cast<const float *>(w)[s.a + i];
            wb[i] = static_cast<const float *>(w)[s.b + i];
        } else {
            wa[i] = float(static_cast<const typename Elem<DT>::type *>(w)[s.a + i]);
            wb[i] = float(static_cast<const typename Elem<DT>::type *>(w)[s.b + i]);
        }
    }
}

// v / scale, cut at the largest e4m3 value: the product with the reciprocal,
// put right by its own remainder.  scale lies between 2^-64 and 2^64.
__device__ __forceinline__ f32x8 over_scale(f32x8 v, float scale)
{
    const float inv = 1.0f / scale, most = 448.0f * scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v[i] != v[i] ? v[i] : fminf(fmaxf(v[i], -most), most);
        const float q = x * inv;
        v[i] = fmaf(fmaf(-q, scale, x), inv, q);
    }
    return v;
}

// Heads [h0, h1) of one token: norm, rotate (TURN), divide by the cache's
// scale, store at dst(h).
template <int DT, int ODT, int LPR, bool ADJ, bool TURN, typename Dst>
__device__ __forceinline__ void turn_heads(const RopeParams &p, const Slot &s, bool on,
                                           const typename Elem<DT>::type *src, const void *weight,
                                           f32x8 cs, f32x8 sn, int h0, int h1, float scale,
                                           Dst dst)
{
    f32x8 wa, wb;
    load_weight<DT>(p, weight, s, wa, wb);
    const float inv_dim = 1.0f / float(p.head_dim);
    for (int h = h0; h < h1; ++h) {
        f32x8 a = 0.0f, b = 0.0f;
        if (on) {
            a = load8<DT>(src + int64_t(h) * p.head_dim + s.a);
            b = load8<DT>(src + int64_t(h) * p.head_dim + s.b);
        }
        if (weight) {
            const float ms = row_sum<LPR>(dot8(a, a) + dot8(b, b)) * inv_dim;
            const float r = 1.0f / sqrtf(ms + p.eps);
            a = a * r * wa;
            b = b * r * wb;
        }
        if constexpr (TURN) rotate<ADJ>(a, b, cs, sn, s.pair >= 0);
        if (!on) continue;
        auto *o = dst(h);
        if constexpr (ODT == kE4M3) {
            a = over_scale(a, scale);
            b = over_scale(b, scale);
        }
        store8<ODT>(o + s.a, a);
        store8<ODT>(o + s.b, b);
    }
}

// grid: (blocks over token groups, head chunks).
template <int DT, int LPR, bool ADJ>
__global__ __launch_bounds__(kBlock) void norm_rope_fwd(RopeParams p, int chunk)
{
    using T = typename Elem<DT>::type;
    constexpr int kRows = kLanes / LPR;
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int wave = int(blockIdx.x) * kWavesPerBlock + int(threadIdx.x) / kLanes;
    const int64_t token = int64_t(wave) * kRows + lane / LPR;
    const Slot s = slot_of(lane % LPR, p.head_dim, p.half, ADJ);
    const bool on = s.on && token < p.n_tokens;
    const int64_t t = token < p.n_tokens ? token : p.n_tokens - 1;
    f32x8 cs, sn;
    angles(p, s, int(t), cs, sn);
    const int h0 = int(blockIdx.y) * chunk;
    const int h1 = min(h0 + chunk, p.n_q_heads + p.n_k_heads);
    if (h0 < p.n_q_heads) {
        T *out = static_cast<T *>(p.q_out) + t * p.q_out_stride;
        turn_heads<DT, DT, LPR, ADJ, true>(p, s, on, static_cast<const T *>(p.q) + t * p.q_stride,
                                     p.q_weight, cs, sn, h0, min(h1, p.n_q_heads), 1.0f,
                                     [&](int h) { return out + int64_t(h) * p.head_dim; });
    }
    if (h1 > p.n_q_heads) {
        T *out = static_cast<T *>(p.k_out) + t * p.k_out_stride;
        turn_heads<DT, DT, LPR, ADJ, true>(p, s, on, static_cast<const T *>(p.k) + t * p.k_stride,
                                     p.k_weight, cs, sn, max(h0 - p.n_q_heads, 0),
                                     h1 - p.n_q_heads, 1.0f,
                                     [&](int h) { return out + int64_t(h) * p.head_dim; });
    }
}

// grid: (blocks over token groups, head chunks); a block walks over token
// groups and leaves one partial row of the weight gradient.  A chunk never
// holds both queries and keys.  Reading the next head before this one is worked
// on costs the registers of a wave a SIMD and loses (16384 tokens of 16 + 4
// heads of 128, forward and backward: 103 us against 101), and so does asking
// for four waves (spills, 313 us).
template <int DT, int LPR, bool ADJ>
__global__ __launch_bounds__(kBlock) void norm_rope_bwd(RopeGradParams g, int chunk, int q_chunks)
{
    using T = typename Elem<DT>::type;
    constexpr int kRows = kLanes / LPR;
    const RopeParams &p = g.rope;
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const Slot s = slot_of(lane % LPR, p.head_dim, p.half, ADJ);
    const bool is_q = int(blockIdx.y) < q_chunks;
    const int heads = is_q ? p.n_q_heads : p.n_k_heads;
    const int h0 = (is_q ? int(blockIdx.y) : int(blockIdx.y) - q_chunks) * chunk;
    const int h1 = min(h0 + chunk, heads);
    const void *weight = is_q ? p.q_weight : p.k_weight;
    f32x8 wa, wb, da = 0.0f, db = 0.0f;
    load_weight<DT>(p, weight, s, wa, wb);
    const float inv_dim = 1.0f / float(p.head_dim);

    const int groups = (p.n_tokens + kRows - 1) / kRows;
    for (int grp = int(blockIdx.x) * kWavesPerBlock + int(threadIdx.x) / kLanes; grp < groups;
         grp += int(gridDim.x) * kWavesPerBlock) {
        const int64_t token = int64_t(grp) * kRows + lane / LPR;
        const bool on = s.on && token < p.n_tokens;
        const int64_t t = token < p.n_tokens ? token : p.n_tokens - 1;
        f32x8 cs, sn;
        angles(p, s, int(t), cs, sn);
        const T *dy = static_cast<const T *>(is_q ? g.dq_out : g.dk_out) +
                      t * (is_q ? g.dq_out_stride : g.dk_out_stride);
        const T *x = static_cast<const T *>(is_q ? p.q : p.k) + t * (is_q ? p.q_stride : p.k_stride);
        T *dx = static_cast<T *>(is_q ? p.q_out : p.k_out) +
                t * (is_q ? p.q_out_stride : p.k_out_stride);
        for (int h = h0; h < h1; ++h) {
            const int64_t row = int64_t(h) * p.head_dim;
            f32x8 ga = 0.0f, gb = 0.0f, xa = 0.0f, xb = 0.0f;
            if (on) {
                ga = load8<DT>(dy + row + s.a);
                gb = load8<DT>(dy + row + s.b);
                if (weight) {
                    xa = load8<DT>(x + row + s.a);
                    xb = load8<DT>(x + row + s.b);
                }
            }
            rotate<ADJ>(ga, gb, cs, -sn, s.pair >= 0);
            if (weight) {
                const float ms = row_sum<LPR>(dot8(xa, xa) + dot8(xb, xb)) * inv_dim;
                // lanes past the last token: their zeros over the root of eps = 0
                // would put NaN into the weight's gradient
                const float r = token < p.n_tokens ? 1.0f / sqrtf(ms + p.eps) : 0.0f;
                xa *= r;
                xb *= r;
                da += ga * xa;
                db += gb * xb;
                ga *= wa;
                gb *= wb;
                const float m = row_sum<LPR>(dot8(ga, xa) + dot8(gb, xb)) * inv_dim;
                ga = (ga - xa * m) * r;
                gb = (gb - xb * m) * r;
            }
            if (on) {
                store8<DT>(dx + row + s.a, ga);
                store8<DT>(dx + row + s.b, gb);
            }
        }
    }
    if (!weight) return;
    // the block's sum of each element: its waves' token rows through LDS, in order
    __shared__ float part[kWavesPerBlock * kRows][LPR * 16];
    float *mine = part[int(threadIdx.x) / LPR];
    if (s.on) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mine[s.a + i] = da[i];
            mine[s.b + i] = db[i];
        }
    }
    __syncthreads();
    const int e = int(threadIdx.x);
    if (e < p.head_dim) {
        float sum = 0.0f;
        for (int i = 0; i < kWavesPerBlock * kRows; ++i) sum += part[i][e];
        g.partials[(int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * p.head_dim + e] = sum;
    }
}

// Sums the partial rows: block (x, 0) the columns 16x.. of dq_weight, (x, 1)
// of dk_weight.  Some hundred rows that wait for memory: 64 strips a block,
// eight loads of each at once (16 strips, one by one: 16 us of the call).
constexpr int kSumBlock = 1024, kStrips = kSumBlock / 16;

__global__ __launch_bounds__(kSumBlock) void sum_partials(const float *partials, int head_dim,
                                                       int q_rows, int k_rows, float *dq_weight,
                                                       float *dk_weight)
{
    const bool is_q = blockIdx.y == 0;
    float *out = is_q ? dq_weight : dk_weight;
    if (!out) return;
    const int rows = is_q ? q_rows : k_rows;
    const float *from = partials + (is_q ? 0 : int64_t(q_rows) * head_dim);
    const int col = int(blockIdx.x) * 16 + int(threadIdx.x) % 16, strip = int(threadIdx.x) / 16;
    float sum = 0.0f;
#pragma unroll 8
    for (int r = strip; r < rows; r += kStrips) sum += from[int64_t(r) * head_dim + col];
    __shared__ float part[kStrips][16];
    part[strip][threadIdx.x % 16] = sum;
    __syncthreads();
    if (strip == 0) {
        for (int i = 1; i < kStrips; ++i) sum += part[i][threadIdx.x % 16];
        out[col] = sum;
    }
}

// grid: (blocks over token groups, head chunks of queries, keys and values).
template <int DT, int CDT, int LPR, bool ADJ>
__global__ __launch_bounds__(kBlock) void append(AppendParams a, int chunk)
{
    using T = typename Elem<DT>::type;
    using C = typename Elem<CDT>::type;
    constexpr int kRows = kLanes / LPR;
    const RopeParams &p = a.rope;
    const PagedParams &g = a.paged;
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int wave = int(blockIdx.x) * kWavesPerBlock + int(threadIdx.x) / kLanes;
    const int64_t first = int64_t(wave) * kRows;
    const int64_t token = first + lane / LPR;
    const bool there = token < p.n_tokens;
    const int64_t t = there ? token : p.n_tokens - 1;
    const Slot s = slot_of(lane % LPR, p.head_dim, p.half, ADJ);

    // the owner of each of the wave's tokens: two searches where one a token
    // took 16384 tokens of one sequence 48.7 us instead of 47.0, 64 of 64
    // sequences 6.6 instead of 5.8
    const auto off = [&](int i) { return int64_t(clip(g.q_offsets[i], 0, p.n_tokens)); };
    int seq = count_upto(g.n_seqs, first, off);
    const int from = seq, more = count_upto(g.n_seqs, first + kRows - 1, off) - from;
    if (more > 0 && more <= kLanes) {            // sequences that end among the wave's tokens
        const int64_t ends = lane < more ? off(from + 1 + lane) : INT64_MAX;
        for (int i = 1; i < kRows; ++i) {
            const int found = from + __popcll(__ballot(ends <= first + i));
            if (lane / LPR == i) seq = found;
        }
    } else if (more != 0) {                      // among them more empty ones than lanes
        for (int i = 1; i < kRows; ++i) {
            const int found = count_upto(g.n_seqs, first + i, off);
            if (lane / LPR == i) seq = found;
        }
    }
    bool owned = there && seq < g.n_seqs;
    const int q = owned ? seq : 0;
    const int begin = int(off(q)), end = int(off(q + 1));
    owned = owned && t >= begin && t < end;
    // the token's slot: its place follows from the length and the end of the
    // sequence as they are, so one past the table is past it here
    const int64_t room = int64_t(g.max_pages) << g.page_shift;
    const int64_t place = int64_t(g.kv_lengths[q]) - g.q_offsets[q + 1] + t;
    int page = -1;
    if (owned && place >= 0 && place < room)
        page = g.block_table[int64_t(q) * g.max_pages + (place >> g.page_shift)];
    const bool kept = page >= 0 && page < g.n_pages;
    const int64_t slot_row = kept ? ((int64_t(page) * p.n_k_heads) << g.page_shift) +
                                        (place & ((1 << g.page_shift) - 1)) : 0;

    f32x8 cs, sn;
    angles(p, s, int(t), cs, sn);
    const int nq = p.n_q_heads, nk = p.n_k_heads;
    const int h0 = int(blockIdx.y) * chunk, h1 = min(h0 + chunk, nq + 2 * nk);
    const bool on = s.on && owned;
    if (h0 < nq) {
        T *out = static_cast<T *>(p.q_out) + t * p.q_out_stride;
        turn_heads<DT, DT, LPR, ADJ, true>(p, s, on, static_cast<const T *>(p.q) + t * p.q_stride,
                                     p.q_weight, cs, sn, h0, min(h1, nq), 1.0f,
                                     [&](int h) { return out + int64_t(h) * p.head_dim; });
    }
    const auto to = [&](void *cache) {
        C *c = static_cast<C *>(cache);
        return [=](int h) {
            return c + (slot_row + (int64_t(h) << g.page_shift)) * p.head_dim;
        };
    };
    const bool keep = on && kept;
    if (h0 < nq + nk && h1 > nq)
        turn_heads<DT, CDT, LPR, ADJ, true>(p, s, keep, static_cast<const T *>(p.k) + t * p.k_stride,
                                      p.k_weight, cs, sn, max(h0 - nq, 0), min(h1 - nq, nk),
                                      g.k_scale, to(g.k_cache));
    if (h1 > nq + nk)
        turn_heads<DT, CDT, LPR, ADJ, false>(p, s, keep, static_cast<const T *>(a.v) + t * a.v_stride,
                                             nullptr, cs, sn, max(h0 - nq - nk, 0), h1 - nq - nk,
                                             g.v_scale, to(g.v_cache));
}

// Heads of one unit of work: enough units for about eight waves for each of
// the 1,024 SIMDs when there are few tokens (six run at once, three to four of
// the gradient's), all heads of a token in one unit (its angles computed once)
// when there are many.
int head_chunk(int64_t token_waves, int heads)
{
    const int64_t want = 8192 / (token_waves > 0 ? token_waves : 1);
    const int64_t chunks = want < 1 ? 1 : (want < heads ? want : heads);
    return int((heads + chunks - 1) / chunks);
}

int lanes_per_row(int head_dim)
{
    int l = 1;
    while (l * 16 < head_dim) l *= 2;
    return l;
}

template <typename F>
void with_lanes(int head_dim, F f)
{
    switch (lanes_per_row(head_dim)) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 8: f(std::integral_constant<int, 8>{}); break;
    default: f(std::integral_constant<int, 16>{}); break;
    }
}

template <typename F>
void with_layout(bool adjacent, F f)
{
    if (adjacent) f(std::true_type{});
    else f(std::false_type{});
}

int64_t blocks_over(int64_t n_tokens, int head_dim)
{
    const int64_t rows = int64_t(kWavesPerBlock) * (kLanes / lanes_per_row(head_dim));
    return (n_tokens + rows - 1) / rows;
}

// Blocks of the gradient kernel over the tokens, and partial rows of q and k.
struct GradGrid { int blocks, chunk, q_chunks, k_chunks; };

GradGrid grad_grid(int64_t n_tokens, int n_q_heads, int n_k_heads, int head_dim)
{
    GradGrid g;
    const int64_t blocks = blocks_over(n_tokens, head_dim);
    g.chunk = head_chunk(blocks * kWavesPerBlock, n_q_heads + n_k_heads);
    g.q_chunks = (n_q_heads + g.chunk - 1) / g.chunk;
    g.k_chunks = (n_k_heads + g.chunk - 1) / g.chunk;
    // blocks the chip holds (2.5 for each CU, by their registers), with equal
    // numbers of token groups: 16384 tokens of 16 + 4 heads of 128, forward and
    // backward, 96 us with 640 or 768, 97 with 1280, 100 with 2560
    const int64_t limit = 640 / (g.q_chunks + g.k_chunks), most = limit > 1 ? limit : 1;
    const int64_t turns = (blocks + most - 1) / most;      // token groups a wave walks over
    g.blocks = int(turns > 0 ? (blocks + turns - 1) / turns : 0);
    return g;
}

}  // namespace

size_t rope_grad_workspace_bytes(int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
                                 int32_t head_dim)
{
    const GradGrid g = grad_grid(n_tokens, n_q_heads, n_k_heads, head_dim);
    const size_t rows = size_t(g.blocks) * (g.q_chunks + g.k_chunks);
    const size_t bytes = rows * head_dim * sizeof(float);
    return bytes < 256 ? 256 : (bytes + 255) & ~size_t(255);
}

hipError_t run_qk_norm_rope(const RopeParams &p, hipStream_t stream)
{
    const int64_t blocks = blocks_over(p.n_tokens, p.head_dim);
    const int heads = p.n_q_heads + p.n_k_heads;
    const int chunk = head_chunk(blocks * kWavesPerBlock, heads);
    const dim3 grid(uint32_t(blocks), uint32_t((heads + chunk - 1) / chunk));
    with_lanes(p.head_dim, [&](auto lpr) {
        with_layout(p.adjacent, [&](auto adj) {
            constexpr int L = decltype(lpr)::value;
            constexpr bool A = decltype(adj)::value;
            switch (p.dtype) {
            case kF32: norm_rope_fwd<kF32, L, A><<<grid, kBlock, 0, stream>>>(p, chunk); break;
            case kF16: norm_rope_fwd<kF16, L, A><<<grid, kBlock, 0, stream>>>(p, chunk); break;
            default: norm_rope_fwd<kBF16, L, A><<<grid, kBlock, 0, stream>>>(p, chunk); break;
            }
        });
    });
    return hipGetLastError();
}

hipError_t run_qk_norm_rope_backward(const RopeGradParams &g, hipStream_t stream)
{
    const RopeParams &p = g.rope;
    const GradGrid w = grad_grid(p.n_tokens, p.n_q_heads, p.n_k_heads, p.head_dim);
    const int blocks = p.n_tokens > 0 ? w.blocks : 0;
    if (blocks > 0) {
        const dim3 grid(uint32_t(blocks), uint32_t(w.q_chunks + w.k_chunks));
        with_lanes(p.head_dim, [&](auto lpr) {
            with_layout(p.adjacent, [&](auto adj) {
                constexpr int L = decltype(lpr)::value;
                constexpr bool A = decltype(adj)::value;
                switch (p.dtype) {
                case kF32:
                    norm_rope_bwd<kF32, L, A><<<grid, kBlock, 0, stream>>>(g, w.chunk, w.q_chunks);
                    break;
                case kF16:
                    norm_rope_bwd<kF16, L, A><<<grid, kBlock, 0, stream>>>(g, w.chunk, w.q_chunks);
                    break;
                default:
                    norm_rope_bwd<kBF16, L, A><<<grid, kBlock, 0, stream>>>(g, w.chunk, w.q_chunks);
                    break;
                }
            });
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!p.q_weight && !p.k_weight) return hipSuccess;
    sum_partials<<<dim3(uint32_t(p.head_dim / 16), 2), kSumBlock, 0, stream>>>(
        g.partials, p.head_dim, blocks * w.q_chunks, blocks * w.k_chunks,
        p.q_weight ? g.dq_weight : nullptr, p.k_weight ? g.dk_weight : nullptr);
    return hipGetLastError();
}

hipError_t run_kv_append(const AppendParams &a, hipStream_t stream)
{
    const RopeParams &p = a.rope;
    const int64_t blocks = blocks_over(p.n_tokens, p.head_dim);
    const int heads = p.n_q_heads + 2 * p.n_k_heads;
    const int chunk = head_chunk(blocks * kWavesPerBlock, heads);
    const dim3 grid(uint32_t(blocks), uint32_t((heads + chunk - 1) / chunk));
    with_lanes(p.head_dim, [&](auto lpr) {
        with_layout(p.adjacent, [&](auto adj) {
            constexpr int L = decltype(lpr)::value;
            constexpr bool A = decltype(adj)::value;
            const bool e4m3 = a.paged.cache_dtype == kE4M3;
            if (p.dtype == kF16 && !e4m3)
                append<kF16, kF16, L, A><<<grid, kBlock, 0, stream>>>(a, chunk);
            else if (p.dtype == kF16)
                append<kF16, kE4M3, L, A><<<grid, kBlock, 0, stream>>>(a, chunk);
            else if (!e4m3)
                append<kBF16, kBF16, L, A><<<grid, kBlock, 0, stream>>>(a, chunk);
            else
                append<kBF16, kE4M3, L, A><<<grid, kBlock, 0, stream>>>(a, chunk);
        });
    });
    return hipGetLastError();
}

}  // namespace bevpool
