// Append to a cache of e4m3 codes with a scale for each block of tokens and head
// (gfx950).  See bevpool.h for the definition; rope_kernels.hip says how head rows
// lie in lanes.
//
// A scale follows from the largest of its block's new rows, so a head's rows are
// read, normed and turned into registers, their largest element is found, and the
// rows leave as codes: one pass over memory.  Where sequences bring few tokens
// (append_heads) the lanes of a wave hold a head's rows and several heads; where they
// bring many (append_blocks) a block of threads holds a block of tokens and walks
// over heads, the waves' largest meeting in LDS, one barrier a head.  1024 threads
// hold 1024 / lanes-per-row tokens at once; wider blocks (256 tokens of 128 dims,
// 128 of 256) are held in two strips, 256 of 256 in four that are read twice.  Their
// angles lie in LDS, so that no register is spilled.
//
// Bound by HBM where large: 16384 tokens of 16 on 8 heads of 128 (bf16, 235 MB)
// 56 us, 4.2 TB/s; what is left to the copy's rate is the begin of each share (offsets,
// lengths and page before the first row) and four waves a SIMD, which is what the
// registers allow (rows, their successors, weights, sines and cosines).  96 single
// tokens 6.8 us: the chain offsets, length, row, page, old scale, code.
//
// Codes of earlier tokens in a block change only where its scale grows.  It grows
// by powers of two, so they stay what they were, but for the bits that leave at
// the bottom of the format.
#include <hip/hip_runtime.h>

#include "append_walk.h"
#include "rope_device.h"

namespace bevpool {
namespace {

constexpr int kMostThreads = 1024, kHeadThreads = 64;
constexpr int kChipThreads = 256 * 1024;      // four waves of append_blocks a SIMD
constexpr float kMostCode = 448.0f;

// The lane's eight angles, in turns from -1/2 to 1/2: formed in fp64, as far positions
// need them.
__device__ __forceinline__ f32x8 fractions(const RopeParams &p, const Slot &s, int token)
{
    f32x8 part = 0.0f;
    if (s.pair < 0) return part;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = s.pair + i;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kMaxRopeAxes - 1; ++a)
            if (a + 1 < p.n_axes && pair >= p.section_end[a]) axis = a + 1;
        const double angle = double(p.positions[int64_t(axis) * p.n_tokens + token]) * double(p.inv_freq[pair]);
        const double per_turn = 0.15915494309189533577;        // 1 / (2 pi)
        part[i] = float(fma(angle, per_turn, -rint(angle * per_turn)));
    }
    return part;
}

// Cosines and sines of four of them, by the hardware's sine, which takes turns and is within
// 2^-22.9 (measured over 2^24 angles; sincospif 2^-24.2, but 40 instructions where
// this is one: 19 prompts of up to 1703 tokens, 10 on 5 heads of 80, 28.0 us with
// that and 26.8 with this).  What comes of it is rounded to 16 bits or to a code.
struct Turn4 { f32x4 cs, sn; };

__device__ __forceinline__ Turn4 turns_of(f32x4 part)
{
    Turn4 t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t.cs[i] = __builtin_amdgcn_cosf(part[i]);
        t.sn[i] = __builtin_amdgcn_sinf(part[i]);
    }
    return t;
}

__device__ __forceinline__ f32x4 low(f32x8 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3); }
__device__ __forceinline__ f32x4 high(f32x8 v) { return __builtin_shufflevector(v, v, 4, 5, 6, 7); }
__device__ __forceinline__ f32x8 both(f32x4 a, f32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// Turns the lane's pairs 0 to 3, or 4 to 7.  Which product a sum takes unrounded is
// written out, here and in the norm: left to the compiler it differed between the
// kernels, and with it a bit of the result between launches.
template <bool ADJ, int HALF>
__device__ __forceinline__ void rotate4(f32x8 &a, f32x8 &b, const Turn4 &t)
{
    f32x8 &own = HALF ? b : a;
    f32x4 u, v;
    if constexpr (ADJ) {
        u = __builtin_shufflevector(own, own, 0, 2, 4, 6);
        v = __builtin_shufflevector(own, own, 1, 3, 5, 7);
    } else {
        u = HALF ? high(a) : low(a);
        v = HALF ? high(b) : low(b);
    }
    const f32x4 x = __builtin_elementwise_fma(u, t.cs, -(v * t.sn)), y = __builtin_elementwise_fma(u, t.sn, v * t.cs);
    if constexpr (ADJ) {
        own = __builtin_shufflevector(x, y, 0, 4, 1, 5, 2, 6, 3, 7);
    } else {
        a = HALF ? both(low(a), x) : both(x, high(a));
        b = HALF ? both(low(b), y) : both(y, high(b));
    }
}

__device__ __forceinline__ float wave_max(float m)
{
#pragma unroll
    for (int i = 1; i < kLanes; i *= 2) m = fmaxf(m, __shfl_xor(m, i));
    return m;
}

// The larger of m and the sizes in v (NaN has none).
__device__ __forceinline__ float size_max(float m, f32x8 v)
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = fmaxf(fmaxf(fabsf(v[i]), fabsf(v[i + 1])), m);
    return m;
}

// The same of those that are finite.
__device__ __forceinline__ float finite_max(float m, f32x8 v)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = fabsf(v[i]);
        m = x < INFINITY ? fmaxf(m, x) : m;
    }
    return m;
}

// The scale of a block whose new rows reach `most`: of a block without earlier
// tokens (old 0) the one that takes it to the largest code; otherwise the old
// one, doubled until it fits.  Whether it fits is a question of one bit, asked
// in fp64, where the product is exact.
__device__ __forceinline__ float scale_for(float most, float old)
{
    if (old == 0.0f) return block_scale(most / kMostCode);
    int e;
    const double m = frexp(double(most) / (double(kMostCode) * double(old)), &e);
    if (m == 0.5) --e;
    return block_scale(ldexpf(old, e > 0 ? e : 0));
}

// v / scale where all of it that is finite is within the largest code and nothing is
// infinite: the product with the reciprocal, put right by its own remainder.
__device__ __forceinline__ f32x8 within_scale(f32x8 v, float scale, float inv)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = v[i] * inv;
        v[i] = fmaf(fmaf(-q, scale, v[i]), inv, q);
    }
    return v;
}

// Four codes times ratio.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio)
{
    return e4m3x4(__builtin_amdgcn_cvt_f32_fp8(int(w), 0) * ratio,
                  __builtin_amdgcn_cvt_f32_fp8(int(w), 1) * ratio,
                  __builtin_amdgcn_cvt_f32_fp8(int(w), 2) * ratio,
                  __builtin_amdgcn_cvt_f32_fp8(int(w), 3) * ratio);
}

// `pieces` 16-byte pieces of codes times ratio, by `lanes` threads, this one the
// n-th; two reads of each at once.
__device__ __forceinline__ void rescale_codes(u32x4 *codes, int pieces, float ratio, int n, int lanes)
{
    for (; n < pieces; n += 2 * lanes) {
        u32x4 c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = n + i * lanes < pieces ? codes[n + i * lanes] : u32x4(0u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (n + i * lanes >= pieces) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) c[i][k] = rescaled(c[i][k], ratio);
            codes[n + i * lanes] = c[i];
        }
    }
}

// The lane's two runs of a head row, as they are.
struct Raw { u32x4 a, b; };

template <int DT>
__device__ __forceinline__ Raw load_raw(const typename Elem<DT>::type *row, const Slot &s, bool on)
{
    Raw r = {u32x4(0u), u32x4(0u)};
    if (on) {
        r.a = *reinterpret_cast<const u32x4 *>(row + s.a);
        r.b = *reinterpret_cast<const u32x4 *>(row + s.b);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ f32x8 floats(u32x4 x)
{
    using V = std::conditional_t<DT == kF16, f16x8, bf16x8>;
    return __builtin_convertvector(__builtin_bit_cast(V, x), f32x8);
}

// Calls f(Piece) for the new tokens of a tile.
template <int PER, typename F>
__device__ __forceinline__ void each_piece(const AppendParams &a, int64_t tile, F f)
{
    const PagedParams &g = a.paged;
    const int seq = count_upto(g.n_seqs, tile, [&](int i) {
        return first_tile<PER>(token_offset(a, i), i, g.block_shift);
    });
    if (seq < g.n_seqs) pieces_of<PER>(a, seq, tile, f);
}

template <int LPR>
__device__ __forceinline__ void normed(f32x8 &x, f32x8 &y, f32x8 wa, f32x8 wb, float inv_dim, float eps)
{
    const float r = 1.0f / sqrtf(fmaf(row_sum<LPR>(dot8(x, x) + dot8(y, y)), inv_dim, eps));
    x = x * r * wa;
    y = y * r * wb;
}

// Few new tokens a block: LPR lanes take a head's row, `together` rows of a head lie
// side by side in a wave, which so has several heads, and a head's largest element
// goes over its lanes.  More tokens than that take turns, and are read twice.
// Earlier codes are rescaled by the wave.
template <int DT, int LPR, bool ADJ>
__global__ __launch_bounds__(kHeadThreads) void append_heads(AppendParams a, int together)
{
    using T = typename Elem<DT>::type;
    const RopeParams &p = a.rope;
    const PagedParams &g = a.paged;
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int nq = p.n_q_heads, nk = p.n_k_heads, heads = nq + 2 * nk;
    const int row_of = (int(blockIdx.y) * kHeadThreads + int(threadIdx.x)) / LPR;
    const int mine = row_of / together, turn = row_of % together, i = min(mine, heads - 1);
    const bool leads = turn == 0 && lane % LPR == 0;        // of the head's lanes
    const bool is_q = i < nq, is_k = !is_q && i < nq + nk;
    const int h = i - (is_q ? 0 : is_k ? nq : nq + nk);
    const Slot s = slot_of(lane % LPR, p.head_dim, p.half, ADJ);
    const bool there = mine < heads;
    const T *src = static_cast<const T *>(is_q ? p.q : is_k ? p.k : a.v) + int64_t(h) * p.head_dim;
    const int64_t stride = is_q ? p.q_stride : is_k ? p.k_stride : a.v_stride;
    const void *weight = is_q ? p.q_weight : is_k ? p.k_weight : nullptr;
    const float inv_dim = 1.0f / float(p.head_dim);

    each_piece<1>(a, blockIdx.x, [&](const Piece &c) {
        const int64_t row = c.row0 + (int64_t(h) << g.page_shift);
        uint8_t *codes = static_cast<uint8_t *>(is_k ? g.k_cache : g.v_cache) + row * p.head_dim;
        float *at = (is_k ? g.k_scales : g.v_scales) + (row >> g.block_shift);
        const bool stored = !is_q && c.kept && there;
        f32x8 x, y;
        const auto take = [&](int t) {
            const bool on = s.on && there && t < c.count;
            t = min(t, c.count - 1);
            const Raw raw = load_raw<DT>(src + (c.token0 + t) * stride, s, on);
            f32x8 wa, wb;
            load_weight<DT>(p, weight, s, wa, wb);
            const f32x8 part = fractions(p, s, int(c.token0 + t));
            x = floats<DT>(raw.a);
            y = floats<DT>(raw.b);
            f32x8 u = x, v = y;
            normed<LPR>(u, v, wa, wb, inv_dim, p.eps);      // by all lanes: it sums over them
            x = weight ? u : x;
            y = weight ? v : y;
            if (s.pair < 0 || !(is_q || is_k)) return;
            rotate4<ADJ, 0>(x, y, turns_of(low(part)));
            rotate4<ADJ, 1>(x, y, turns_of(high(part)));
        };
        const float old = stored && c.early > 0 ? block_scale(*at) : 0.0f;
        float most = 0.0f;
        for (int t = turn; t < c.count + turn; t += together) {
            take(t);
            most = finite_max(finite_max(most, x), y);
        }
        for (int m = 1; m < LPR * together; m *= 2) most = fmaxf(most, __shfl_xor(most, m));
        const float scale = scale_for(most, old);
        for (int t = turn; t < c.count + turn; t += together) {
            if (c.count > together) take(t);
            if (!s.on || !there || t >= c.count) continue;
            if (is_q) {
                T *out = static_cast<T *>(p.q_out) + (c.token0 + t) * p.q_out_stride + int64_t(h) * p.head_dim;
                store8<DT>(out + s.a, x);
                store8<DT>(out + s.b, y);
            } else if (stored) {
                uint8_t *out = codes + int64_t(c.early + t) * p.head_dim;
                store8<kE4M3>(out + s.a, over_scale(x, scale));
                store8<kE4M3>(out + s.b, over_scale(y, scale));
            }
        }
        if (stored && leads) *at = scale;
        uint64_t grown = __ballot(stored && c.early > 0 && scale != old && leads);
        while (grown) {
            const int from = __builtin_ctzll(grown);
            grown &= grown - 1;
            uint8_t *base = static_cast<uint8_t *>(__shfl(int(is_k), from) ? g.k_cache : g.v_cache);
            rescale_codes(reinterpret_cast<u32x4 *>(base + __shfl(row, from) * p.head_dim),
                          c.early * p.head_dim / 16, __shfl(old / scale, from), lane, kLanes);
        }
    });
}

// Many: a head at a time, its rows dealt to the threads, the next head's on their
// way while this one is worked on.  The heads of all tiles (queries, keys, values)
// go in equal shares to as many blocks as the chip holds.  (A grid of tiles and
// quarters of the heads takes 53 us instead of 56 for 16384 tokens of 16 on 8 heads
// of 128 where its blocks are two to a CU, 58 where one more tile makes them a few
// more, and 75 with halves of the heads.)  blockDim.x / LPR rows a strip.
template <int DT, int LPR, bool ADJ, int STRIPS>
__global__ __launch_bounds__(kMostThreads) void append_blocks(AppendParams a, int64_t units)
{
    using T = typename Elem<DT>::type;
    constexpr bool kHold = STRIPS <= 2;
    constexpr bool kAhead = STRIPS == 1;            // registers for more are not there
    constexpr int kHeld = kHold ? STRIPS : 1;
    __shared__ float wave_most[2][kMostThreads / kLanes];
    // Of several strips' angles: two strips' sines and cosines, four strips' turns; a
    // thread reads what it wrote.
    constexpr int kPieces = STRIPS == 1 ? 0 : 8 / STRIPS;
    __shared__ f32x4 angles_of[STRIPS == 1 ? 1 : 8 * kMostThreads];
    const RopeParams &p = a.rope;
    const PagedParams &g = a.paged;
    const int tid = int(threadIdx.x), lane = tid & (kLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kLanes);
    const int rows = int(blockDim.x) / LPR;
    const int nq = p.n_q_heads, nk = p.n_k_heads, heads = nq + 2 * nk;
    const float inv_dim = 1.0f / float(p.head_dim);
    const int64_t first = units * blockIdx.x / gridDim.x, last = units * (blockIdx.x + 1) / gridDim.x;

    for (int64_t at = first, tile = first / heads; at < last; at = ++tile * heads) {
        const int h0 = int(at - tile * heads), h1 = int(min(last - tile * heads, int64_t(heads)));
        // what follows from the lane is worked out for each tile: kept from one to
        // the next it would take the registers that hold rows
        int j = lane % LPR;
        asm volatile("" : "+v"(j));
        const Slot s = slot_of(j, p.head_dim, p.half, ADJ);
        if (at > first) __syncthreads();         // the last tile's sizes have been read
        each_piece<2>(a, tile, [&](const Piece &c) {
            const int waves = (min(c.count, rows) * LPR + kLanes - 1) / kLanes;     // that have rows
            const auto index = [&](int st) { return st * rows + tid / LPR; };
            const auto on = [&](int st) { return s.on && index(st) < c.count; };
            const auto token = [&](int st) { return c.token0 + index(st); };        // where on(st)
            const auto used = [&](int st) { return st == 0 || st * rows < c.count; };
            Turn4 held[2];
            f32x8 wa, wb;
            const auto piece = [&](int st, int n) -> f32x4 & {
                return angles_of[(st * kPieces + n) * kMostThreads + tid];
            };
            if (h0 < nq + nk) {
                for (int st = 0; st < STRIPS; ++st) {
                    if (!used(st)) continue;
                    const f32x8 part = fractions(p, s, int(c.token0) + min(index(st), c.count - 1));
                    if constexpr (STRIPS == 4) {
                        piece(st, 0) = low(part);
                        piece(st, 1) = high(part);
                    } else {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const Turn4 t = turns_of(n ? high(part) : low(part));
                            if constexpr (STRIPS == 1) {
                                held[n] = t;
                            } else {
                                piece(st, 2 * n) = t.cs;
                                piece(st, 2 * n + 1) = t.sn;
                            }
                        }
                    }
                }
            }
            const auto turn4 = [&](int st, int n) {
                if constexpr (STRIPS == 1) return held[n];
                else if constexpr (STRIPS == 2) return Turn4{piece(st, 2 * n), piece(st, 2 * n + 1)};
                else return turns_of(piece(st, n));
            };
            // Heads [from, to) of one kind, each as fetched, normed and turned.
            Raw next;
            const auto fetch = [&](const void *src, int64_t stride, int h, int st) {
                return load_raw<DT>(static_cast<const T *>(src) + token(st) * stride + int64_t(h) * p.head_dim, s, on(st));
            };
            const auto take = [&](int st, Raw raw, bool norm, bool turn, f32x8 &x, f32x8 &y) {
                x = floats<DT>(raw.a);
                y = floats<DT>(raw.b);
                if (norm) normed<LPR>(x, y, wa, wb, inv_dim, p.eps);
                if (!turn || s.pair < 0) return;
                rotate4<ADJ, 0>(x, y, turn4(st, 0));
                rotate4<ADJ, 1>(x, y, turn4(st, 1));
            };

            if (h0 < nq && (waves > 1 || wave == 0)) {
                const int to = min(h1, nq);
                if (kAhead) next = fetch(p.q, p.q_stride, h0, 0);
                load_weight<DT>(p, p.q_weight, s, wa, wb);
                for (int h = h0; h < to; ++h) {
#pragma unroll
                    for (int st = 0; st < STRIPS; ++st) {
                        if (!used(st)) continue;
                        const Raw raw = kAhead ? next : fetch(p.q, p.q_stride, h, st);
                        if (kAhead && h + 1 < to) next = fetch(p.q, p.q_stride, h + 1, 0);
                        f32x8 x, y;
                        take(st, raw, p.q_weight, true, x, y);
                        if (!on(st)) continue;
                        T *out = static_cast<T *>(p.q_out) + token(st) * p.q_out_stride + int64_t(h) * p.head_dim;
                        store8<DT>(out + s.a, x);
                        store8<DT>(out + s.b, y);
                    }
                }
            }
            const auto store = [&](const void *src, int64_t stride, bool norm, bool turn, void *cache, float *scales,
                                   int from, int to) {
                if (kAhead && from < to) next = fetch(src, stride, from, 0);
                for (int h = from; h < to; ++h) {
                    const int64_t row = c.row0 + (int64_t(h) << g.page_shift);
                    uint8_t *codes = static_cast<uint8_t *>(cache) + row * p.head_dim;
                    float *at = scales + (row >> g.block_shift);
                    const float old = c.early > 0 ? block_scale(*at) : 0.0f;
                    f32x8 x[kHeld], y[kHeld];
                    float most = 0.0f;
                    bool cut = false;
#pragma unroll
                    for (int st = 0; st < STRIPS; ++st) {
                        if (!used(st)) continue;
                        const int n = kHold ? st : 0;
                        const Raw raw = kAhead ? next : fetch(src, stride, h, st);
                        if (kAhead && h + 1 < to) next = fetch(src, stride, h + 1, 0);
                        take(st, raw, norm, turn, x[n], y[n]);
                        float m = size_max(size_max(0.0f, x[n]), y[n]);
                        if (__any(m == INFINITY)) {
                            m = finite_max(finite_max(0.0f, x[n]), y[n]);
                            cut = true;
                        }
                        most = fmaxf(most, m);
                    }
                    most = wave_max(most);
                    if (waves > 1) {
                        float *all = wave_most[h & 1];
                        if (lane == 0) all[wave] = most;
                        asm volatile("" : : "v"(old));      // is there before the first thread writes the new one
                        __syncthreads();
                        for (int w = 0; w < waves; ++w) most = fmaxf(most, all[w]);
                    }
                    const float scale = scale_for(most, old), inv = 1.0f / scale;
                    cut |= scale == kMostBlockScale;
                    if (tid == 0) *at = scale;
                    if (c.early > 0 && scale != old && wave < waves)
                        rescale_codes(reinterpret_cast<u32x4 *>(codes), c.early * p.head_dim / 16, old / scale, tid,
                                      waves * kLanes);
#pragma unroll
                    for (int st = 0; st < STRIPS; ++st) {
                        if (!used(st)) continue;
                        const int n = kHold ? st : 0;
                        if (!kHold) take(st, fetch(src, stride, h, st), norm, turn, x[0], y[0]);
                        if (!on(st)) continue;
                        uint8_t *out = codes + int64_t(c.early + index(st)) * p.head_dim;
                        if (cut) {
                            x[n] = over_scale(x[n], scale);
                            y[n] = over_scale(y[n], scale);
                        } else {
                            x[n] = within_scale(x[n], scale, inv);
                            y[n] = within_scale(y[n], scale, inv);
                        }
                        store8<kE4M3>(out + s.a, x[n]);
                        store8<kE4M3>(out + s.b, y[n]);
                    }
                }
                // the last head's sizes are read before the next kind's are written
                if (waves > 1 && from < to) __syncthreads();
            };
            if (!c.kept || h1 <= nq || (waves == 1 && wave > 0)) return;
            load_weight<DT>(p, p.k_weight, s, wa, wb);
            store(p.k, p.k_stride, p.k_weight, true, g.k_cache, g.k_scales, max(h0 - nq, 0), min(h1 - nq, nk));
            store(a.v, a.v_stride, false, false, g.v_cache, g.v_scales, max(h0 - nq - nk, 0), h1 - nq - nk);
        });
    }
}

struct Launch {
    int together;          // rows of append_heads; 0: append_blocks
    int threads, strips;
    int64_t tiles, waves;  // waves of append_heads for a tile
};

Launch launch_of(int64_t n_tokens, int32_t n_seqs, int64_t heads, int32_t head_dim, int32_t block_shift)
{
    Launch l = {};
    const int lanes = lanes_per_row(head_dim), rows = kLanes / lanes;
    // Up to twice a wave's rows a sequence, on average.  64 sequences of 32 + 16 heads
    // of 128, blocks of 64: two new tokens 6.9 us so and 22 by append_blocks, eight
    // 11.2 and 24, 16 27.9 and 32.4, 32 46 and 35.
    if (n_tokens <= 2 * rows * int64_t(n_seqs)) {
        l.together = 1;
        while (l.together < rows && l.together * int64_t(n_seqs) < n_tokens) l.together *= 2;
        l.threads = kHeadThreads;
        l.tiles = (n_tokens >> block_shift) + n_seqs;
        l.waves = (heads * l.together * lanes + kLanes - 1) / kLanes;
        // a grid has 2^32 threads one way and 65535 blocks the other
        if (l.tiles * kHeadThreads <= UINT32_MAX && l.waves <= 65535) return l;
        l.together = 0;
    }
    const int all = lanes << block_shift;
    l.threads = all < kLanes ? kLanes : all < kMostThreads ? all : kMostThreads;
    l.strips = all > kMostThreads ? all / kMostThreads : 1;
    l.tiles = (n_tokens >> block_shift) + 2 * int64_t(n_seqs);
    return l;
}

}  // namespace

hipError_t run_kv_append_scaled(const AppendParams &a, hipStream_t stream)
{
    const RopeParams &p = a.rope;
    const int heads = p.n_q_heads + 2 * p.n_k_heads;
    const Launch l = launch_of(p.n_tokens, a.paged.n_seqs, heads, p.head_dim, a.paged.block_shift);
    const int64_t units = l.tiles * heads, room = kChipThreads / l.threads;
    const uint32_t grid = uint32_t(units < room ? units : room);
    const dim3 few(uint32_t(l.tiles), uint32_t(l.waves));
    with_lanes(p.head_dim, [&](auto lpr) {
        with_layout(p.adjacent, [&](auto adj) {
            constexpr int L = decltype(lpr)::value;
            constexpr bool A = decltype(adj)::value;
            if (l.together) {
                if (p.dtype == kF16) append_heads<kF16, L, A><<<few, kHeadThreads, 0, stream>>>(a, l.together);
                else append_heads<kBF16, L, A><<<few, kHeadThreads, 0, stream>>>(a, l.together);
                return;
            }
            const auto go = [&](auto strips) {
                constexpr int S = decltype(strips)::value;
                if (p.dtype == kF16) append_blocks<kF16, L, A, S><<<grid, l.threads, 0, stream>>>(a, units);
                else append_blocks<kBF16, L, A, S><<<grid, l.threads, 0, stream>>>(a, units);
            };
            // blocks have up to 256 tokens
            if constexpr (L == 16) {
                if (l.strips == 4) return go(std::integral_constant<int, 4>{});
            }
            if constexpr (L >= 8) {
                if (l.strips == 2) return go(std::integral_constant<int, 2>{});
            }
            go(std::integral_constant<int, 1>{});
        });
    });
    return hipGetLastError();
}

}  // namespace bevpool
