// Attention over a paged cache (gfx950).  See bevpool.h for the definition.
//
// The query heads that share a key head are rows of one product: the rows of
// a (sequence, key head) are r = token * G + g, G = n_q_heads / n_k_heads.  A
// block of eight waves takes a tile of consecutive rows and a range of keys.
// A wave owns 32 rows; with 256 rows in a tile the waves walk the keys
// together, with 128 four of them take every other 64 keys, and with 32 or
// fewer each takes every eighth 32 keys; waves with the same rows join at the
// end, in LDS.  Ranges of keys are cut over blocks when tiles alone do not
// fill the chip, and attend_join adds their parts.  (Heads over 128 wide fill
// a wave's registers: their blocks have four waves and 128 rows.)
//
// Both products run on 32 x 32 x 16 matrix instructions, transposed:
//     S^T [keys x rows] = K Q^T,      O^T [dim x rows] += V^T P^T,
// so a row of the softmax is a column of the result: a lane holds 16 of its
// column's 32 keys, its maximum and sum need one exchange between the two
// halves of the wave, and rescaling O is a multiplication by a lane's own
// scalar.  The result registers of S^T hold keys 8 (i / 4) + 4 half + i % 4;
// taken as the second product's inner index in that order they are its
// operand as they stand, and V^T is read from LDS in the same order by the
// transposing read (four keys of one dim a lane), so the weights never leave
// their registers.
//
// What bounds it.  Single tokens read each key and value once: 64 requests of
// up to 8192 keys (32 heads on 8, 128 dims, bf16) 245 us, 5.6 TB/s; two of
// 131072 (e4m3) 47 us and 7 for the join.  Chunks are bound by issue: for 64
// keys of 128 dims a wave has 32 matrix instructions (1024 cycles of the
// matrix cores), 32 exponentials and some 200 other vector instructions, and
// the two waves of a SIMD take about 4200 cycles for theirs: the matrix cores
// are busy 46 % of the time.  4096 tokens after 8192 cached ones (32 heads on 8)
// take 670 to 700 us in a row, 0.98 to 1.03 PFLOP/s, and 730 to 840 in a
// profiler's pauses, at the clock that power leaves (2.3 GHz falling to 1.7);
// the library's large product reaches 1.18.  A block takes about 13 us to begin
// (its place, its queries, its first keys) and end: a sixth of 6 x 704 tokens
// over 2816 keys (80 dims, 77 to 86 us), which keep 144 of the 256 CUs.
#include <hip/hip_runtime.h>

#include "token_device.h"

namespace bevpool {
namespace {

constexpr int kRowsPerWave = 32;
constexpr int kUnit = 256;            // keys: ranges of a split are multiples of this
constexpr float kLog2e = 1.44269504088896340736f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int16_t i16x4 __attribute__((ext_vector_type(4)));

// Type in which keys meet queries, and values meet weights.  e4m3 widens
// exactly to either 16-bit type; fp16 rounds the weights 8 times finer.
template <int DT, int CDT> struct Types { static constexpr int V = CDT == kE4M3 ? int(kF16) : DT; };

// Weights, and so their sums, are 2^lift times what the reference makes them:
// at most 2^15 (the reference may lie 2^8 low), inside fp16, which otherwise
// would round those under 2^-25 to 0, however many there are; so it does those
// under 2^-32.  The factor leaves with the division by the sum.
template <int VT> constexpr float lift() { return VT == kF16 ? 7.0f : 0.0f; }

template <int DT> struct Frag;
template <> struct Frag<kF16> { using type = f16x8; };
template <> struct Frag<kBF16> { using type = bf16x8; };

template <int DT>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
{
    using F = typename Frag<DT>::type;
    if constexpr (DT == kF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(F, a),
                                                      __builtin_bit_cast(F, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(F, a),
                                                       __builtin_bit_cast(F, b), c, 0, 0, 0);
}

// LDS tiles: key and value rows one after the other, in 16-byte pieces, with
// the pieces of a row permuted (a direct load to LDS writes consecutive
// addresses, so rows cannot be padded).  Keys: a phase of a 16-byte read
// takes one piece of 16 consecutive keys; the permutation sends those to 16
// different bank groups.  Values: a phase of a transposing read takes 64
// bytes of four consecutive keys; they go to four different quarters of the
// 256 bytes of banks (a row of 10 pieces shares a few).
template <int DP> struct Tiles {
    static constexpr int kSteps = DP / 16;                 // inner steps of K Q^T
    static constexpr int kDims = (DP + 31) / 32;           // 32-row pieces of O^T
    static constexpr int kPieces = DP / 8;                 // 16-byte pieces of a row
    static constexpr int kRow = DP * 2;
    static constexpr int kRound = kPieces & -kPieces;      // largest power of 2 in kPieces
    static constexpr int kSpread = kRound < 16 ? kRound : 16;
    static constexpr int kWaves = DP > 128 ? 4 : 8;        // of a block
    static constexpr int kBuffers = kWaves * 2 * 32 * kRow;     // keys and values of 32 for each
    static constexpr int kSumRow = DP + 4;                 // floats of a row on the way out
    static constexpr int kSums = kWaves * 32 * kSumRow * 4;
    // room past the last row: the last 32-dim piece of a 16-dim remainder reads it
    static constexpr int kLds = (kBuffers > kSums ? kBuffers : kSums) + 64;

    static __device__ __forceinline__ int key_swizzle(int key)
    {
        return (key / (16 / kSpread)) & (kSpread - 1);
    }
    static __device__ __forceinline__ int value_swizzle(int key)
    {
        if constexpr (kPieces % 16 == 0) return (key & 3) << 2;
        else if constexpr (kPieces % 8 == 0) return ((key >> 1) & 1) << 2;
        else return 0;
    }
};

// What a block works on.
struct Plan {
    int seq, begin, q_len;     // sequence, its first token, its new tokens
    int len;                   // its cached tokens, at most the table's
    int64_t place0;            // place of its first token, from lengths and offsets as they are
    int row0, rows;            // first row of the tile, rows in it
    int lo, hi;                // keys any of them sees: [lo, hi), lo a multiple of 64
    int per;                   // keys of one split
    int splits;                // splits that have keys (at least 1)
};

__device__ __forceinline__ void row_limits(const AttnParams &p, const Plan &w, int row, int group,
                                           int &lo, int &hi)
{
    const int64_t place = w.place0 + row / group;
    int64_t h = p.causal ? place + 1 : w.len, l = p.window > 0 ? place - p.window + 1 : 0;
    h = h < 0 ? 0 : (h > w.len ? w.len : h);
    l = l < 0 ? 0 : (l > w.len ? w.len : l);
    lo = int(l);
    hi = int(h);
}

// Fills in everything of w that follows from seq, begin, q_len, len, row0.
__device__ __forceinline__ void plan_keys(const AttnParams &p, Plan &w, int group, int tile_rows, int max_splits)
{
    const int left = w.q_len * group - w.row0;
    w.rows = left < tile_rows ? left : tile_rows;
    int lo, hi, unused;
    row_limits(p, w, w.row0, group, lo, unused);
    row_limits(p, w, w.row0 + w.rows - 1, group, unused, hi);
    w.lo = lo & ~63;
    w.hi = hi > w.lo ? hi : w.lo;
    const int units = (w.hi - w.lo + kUnit - 1) / kUnit;
    int per = (units + max_splits - 1) / max_splits;
    per = per < 1 ? 1 : per;
    w.per = per * kUnit;
    w.splits = units > per ? (units + per - 1) / per : 1;
}

__device__ __forceinline__ void plan_sequence(const AttnParams &p, Plan &w, int seq, int begin, int end)
{
    const PagedParams &g = p.paged;
    const int64_t room = int64_t(g.max_pages) << g.page_shift;
    const int len = g.kv_lengths[seq];
    w.seq = seq;
    w.begin = begin;
    w.q_len = end - begin;
    w.len = len < 0 ? 0 : (len < room ? len : int(room));
    w.place0 = int64_t(len) - g.q_offsets[seq + 1] + begin;
}

// The sequence and first row of a tile, by the whole wave.  The tiles of
// sequence s start at off(s) * G / tile_rows + s: each has room for all of its rows,
// and the start grows with s.  Fills in w up to row0; false for a tile that is
// nobody's.
__device__ __forceinline__ bool find_tile(const AttnParams &p, Plan &w, int tile, int group,
                                          int tile_rows)
{
    const PagedParams &g = p.paged;
    const auto off = [&](int i) { return clip(g.q_offsets[i], 0, p.n_tokens); };
    const auto start = [&](int i) { return int64_t(off(i)) * group / tile_rows + i; };
    const int seq = count_upto(g.n_seqs, tile, start);
    if (seq >= g.n_seqs) return false;
    const int begin = off(seq), end = off(seq + 1);
    const int64_t row0 = (tile - start(seq)) * tile_rows;
    if (row0 < 0 || row0 >= int64_t(end - begin) * group) return false;
    plan_sequence(p, w, seq, begin, end);
    w.row0 = int(row0);
    return true;
}

// One wave's rows: their part of O^T, the reference maximum of the scores
// (before the scale) with what follows from it, and this lane's part of the
// weights' sum.
template <int DP> struct Rows {
    f32x16 o[Tiles<DP>::kDims];
    float top, base, limit;     // reference; what exponents are told from; past this it moves
    float sum;

    __device__ Rows() : top(-INFINITY), base(0.0f), limit(-INFINITY), sum(0.0f)
    {
#pragma unroll
        for (int dt = 0; dt < Tiles<DP>::kDims; ++dt) o[dt] = 0.0f;
    }
};

// 16-bit values with all exponent bits set (infinity, NaN) in a dword pair.
template <int VT>
__device__ __forceinline__ bool non_finite(u32x4 v)
{
    constexpr uint32_t m = VT == kF16 ? 0x7c00u : 0x7f80u;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (v[i] & m) == m || ((v[i] >> 16) & m) == m;
    return bad;
}

template <int VT>
__device__ __forceinline__ u32x4 finite_only(u32x4 v)
{
    constexpr uint32_t m = VT == kF16 ? 0x7c00u : 0x7f80u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t x = v[i];
        if ((x & m) == m) x &= 0xffff0000u;
        if (((x >> 16) & m) == m) x &= 0xffffu;
        v[i] = x;
    }
    return v;
}

// Eight e4m3 codes as DT (exact).
template <int DT>
__device__ __forceinline__ u32x4 widen(u32x2 raw)
{
    if constexpr (DT == kF16) {
        const int a = int(raw.x), b = int(raw.y);
        u32x4 w;
        w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false));
        w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true));
        w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false));
        w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true));
        return w;
    } else {
        const int a = int(raw.x), b = int(raw.y);
        u32x4 w;
        w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false));
        w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true));
        w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false));
        w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true));
        return w;
    }
}

__device__ const u32x4 kZeroPiece = {0, 0, 0, 0};

// One 16-byte piece for each lane, straight from memory to LDS: lane i's goes
// to LDS address at + 16 i.  Not seen by the compiler's wait counts: a
// wait_loads<n> before the data is used is the caller's.  An M0 write and the
// load that uses it need a wait state between them.
__device__ __forceinline__ void load_to_lds(const void *from, uint32_t at)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(from), "s"(at)
                 : "memory", "m0");
}

// The same from a uniform base and a lane's byte offset.
__device__ __forceinline__ void load_to_lds(const void *base, uint32_t offset, uint32_t at)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %0"
                 :
                 : "s"(base), "v"(offset), "s"(at)
                 : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_address(const char *p)
{
    return __builtin_amdgcn_readfirstlane(
        uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)p)));
}

// Waits until at most N of the wave's memory reads are pending (they complete
// in order).
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// Brings tiles of keys to LDS.  The keys of a tile are 16-key groups, each on
// one page; lane i of a wave keeps the place in the cache of the i-th group to
// come, 64 groups at a time.  Groups on no page, or outside [begin, end), are
// read from page 0 and hidden later, so every read is inside the cache.
//
// A tile of 64 keys is shared by WAVES waves (four: a group each, eight: half
// of one); with WAVES = 1 a tile of 32 is a wave's own.  16-bit caches go
// straight to LDS, e4m3 ones are read into registers (fetch) and widened on
// the way to LDS (store).  AHEAD: the tile is the last 32 keys of one stride
// and the first 32 of the next.
template <int DT, int CDT, int DP, bool EXACT, int WAVES, bool AHEAD>
struct Stage {
    using L = Tiles<DP>;
    using C = typename Elem<CDT>::type;
    static constexpr int VT = Types<DT, CDT>::V;
    static constexpr bool kDirect = CDT != kE4M3;
    static constexpr int kGroups = WAVES > 1 ? 4 : 2;
    static constexpr int kMine = WAVES > 1 ? 1 : 2;                 // groups a wave reads of
    static constexpr int kParts = (L::kPieces + 3) / 4;             // 64-lane loads of a group,
    static constexpr bool kHalfPart = L::kPieces % 4 != 0;          // the last one of 32 lanes
    static constexpr int kHalves = WAVES == 8 ? 2 : 1;              // waves that share a group
    static constexpr int kSlots = (kParts + kHalves - 1) / kHalves; // a wave's loads of a group,
    static constexpr int kLoads = kMine * kSlots;                   // of a tile
    static constexpr int kBatch = kLanes / kGroups;                 // tiles of a batch of groups
    static constexpr int kGroupBytes = 16 * L::kRow;

    const AttnParams &p;
    const int32_t *table;
    int kv_head, wave, begin, end;             // keys [begin, end) are wanted
    int first, stride;                         // tile t holds keys first + t * stride ...
    int row_bytes;
    uint32_t group_lo, group_hi;               // lane's group: its byte offset in the cache
    uint64_t have;                             // groups that are on a page
    // Where rows have a power of two of pieces, the swizzle of a later load is
    // that of the first with some bits turned: registers for all of them would
    // spill in wide heads, and each reload waits for the reads in flight (2 x 1024
    // tokens over 4096 keys, 16 heads of 256 on 4, bf16: 348 -> 269 us).
    static constexpr bool kOne = EXACT && kHalves == 1 && L::kRound == L::kPieces;
    int offset[2][kOne ? 1 : kSlots];          // lane's pieces: bytes from their group, -1 for a zero
    u32x2 k[kDirect ? 1 : kLoads], v[kDirect ? 1 : kLoads];

    __device__ Stage(const AttnParams &p, const Plan &w, int kv_head, int wave, int first,
                     int stride, int begin, int end)
        : p(p), table(p.paged.block_table + int64_t(w.seq) * p.paged.max_pages), kv_head(kv_head),
          wave(wave), begin(begin), end(end), first(first), stride(stride),
          row_bytes(p.head_dim * int(sizeof(C)))
    {
#pragma unroll
        for (int n = 0; n < (kOne ? 1 : kSlots); ++n) {
            const int id = part(n) * kLanes + (int(threadIdx.x) & (kLanes - 1));
            const int key = id / L::kPieces, at = id % L::kPieces;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int piece = at ^ (i ? L::value_swizzle(key) : L::key_swizzle(key));
                offset[i][n] = piece * 8 < p.head_dim
                                   ? key % 16 * row_bytes + piece * 8 * int(sizeof(C)) : -1;
            }
        }
    }

    __device__ __forceinline__ void find_pages(int tile)
    {
        const PagedParams &g = p.paged;
        const int lane = int(threadIdx.x) & (kLanes - 1);
        int group = lane % kGroups, later = 0;
        if (AHEAD) {
            later = group / 2;
            group ^= 2;
        }
        const int64_t key = first + int64_t(tile + lane / kGroups + later) * stride + group * 16;
        int page = -1;
        if (key >= begin && key < end) page = table[key >> g.page_shift];
        if (page >= g.n_pages) page = -1;
        have = __ballot(page >= 0);
        const int64_t row = ((int64_t(max(page, 0)) * p.n_k_heads + kv_head) << g.page_shift) +
                            (key & ((1 << g.page_shift) - 1));
        const uint64_t at = uint64_t(row) * uint32_t(row_bytes);
        group_lo = uint32_t(at);
        group_hi = uint32_t(at >> 32);
    }

    // One bit for each 16-key group of the tile that is on a page.
    __device__ __forceinline__ uint32_t groups_there(int tile) const
    {
        return uint32_t(have >> (tile % kBatch * kGroups)) & ((1u << kGroups) - 1);
    }

    // The part of a group that this wave's load n brings, and whether the lane
    // has a piece of it.
    __device__ __forceinline__ int part(int n) const { return n * kHalves + (kHalves > 1 ? wave / 4 : 0); }
    __device__ __forceinline__ bool has_piece(int n) const
    {
        if constexpr (kParts % kHalves == 0 && !kHalfPart) return true;
        else return part(n) * kLanes + (int(threadIdx.x) & (kLanes - 1)) < 16 * L::kPieces;
    }

    template <bool VALUES> __device__ __forceinline__ int offset_of(int n) const
    {
        if constexpr (kOne) {
            const int key = n * kLanes / L::kPieces;
            const int turned = VALUES ? L::value_swizzle(key) : L::key_swizzle(key);
            return (offset[VALUES][0] ^ (turned * 8 * int(sizeof(C)))) + key * DP * int(sizeof(C));
        } else {
            return offset[VALUES][n];
        }
    }

    // Where the wave's i-th group of a tile lies in a cache.
    __device__ __forceinline__ const char *group_at(const void *cache, int tile, int i) const
    {
        const int lane = tile % kBatch * kGroups + (WAVES > 1 ? wave % 4 : i);
        const uint64_t lo = uint32_t(__builtin_amdgcn_readlane(int(group_lo), lane));
        const uint64_t hi = uint32_t(__builtin_amdgcn_readlane(int(group_hi), lane));
        return static_cast<const char *>(cache) + (hi << 32 | lo);
    }

    // Issues load n of the wave's i-th group, of keys or of values, to the
    // tile at LDS address lds.
    template <bool VALUES>
    __device__ __forceinline__ void fetch_part(const char *base, int i, int n, uint32_t lds)
    {
        const uint32_t to = lds + (WAVES > 1 ? wave % 4 : i) * kGroupBytes + part(n) * 1024;
        const int off = offset_of<VALUES>(n);
        if constexpr (kDirect) {
            if (!has_piece(n)) return;
            if constexpr (EXACT) load_to_lds(base, uint32_t(off), to);
            else load_to_lds(off < 0 ? reinterpret_cast<const char *>(&kZeroPiece) : base + off, to);
        } else {
            // in wide heads, an address made here: with the same load on two
            // paths, the addresses of all would otherwise be kept, and spill
            if constexpr (DP > 128) asm volatile("" : "+s"(base));
            u32x2 x = 0u;
            if (has_piece(n) && (EXACT || off >= 0)) x = *reinterpret_cast<const u32x2 *>(base + uint32_t(off));
            (VALUES ? v : k)[i * kSlots + n] = x;
        }
    }

    template <bool VALUES>
    __device__ __forceinline__ void fetch(int tile, uint32_t lds)
    {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const char *base = group_at(VALUES ? p.paged.v_cache : p.paged.k_cache, tile, i);
#pragma unroll
            for (int n = 0; n < kSlots; ++n) fetch_part<VALUES>(base, i, n, lds);
        }
    }

    // Calls f(byte in the tile, key, register) for each of this lane's pieces.
    template <typename F>
    __device__ __forceinline__ void each_piece(F f) const
    {
        const int lane = int(threadIdx.x) & (kLanes - 1);
#pragma unroll
        for (int i = 0; i < kMine; ++i)
#pragma unroll
            for (int n = 0; n < kSlots; ++n) {
                if (!has_piece(n)) continue;
                const int id = part(n) * kLanes + lane, group = WAVES > 1 ? wave % 4 : i;
                f(group * kGroupBytes + id * 16, group * 16 + id / L::kPieces, i * kSlots + n);
            }
    }

    // e4m3: what fetch read, widened, to LDS.
    template <bool VALUES>
    __device__ __forceinline__ void store(char *lds)
    {
        if constexpr (!kDirect)
            each_piece([&](int at, int, int n) {
                *reinterpret_cast<u32x4 *>(lds + at) = widen<VALUES ? VT : DT>((VALUES ? v : k)[n]);
            });
    }

    // Of the pieces this wave has read, before the others see them: values of
    // places that no row sees become zeros (the tail of a
    // page may hold anything, and 0 * NaN is not 0); so do infinities and NaN
    // that some rows see and others do not, whose first and last key bad gets.
    __device__ __forceinline__ void clean_values(char *lds, int tile, uint32_t there, int *bad) const
    {
        const int key0 = first + tile * stride;
        each_piece([&](int at, int key, int) {
            u32x4 *x = reinterpret_cast<u32x4 *>(lds + at);
            if (key0 + key >= end || !((there >> (key / 16)) & 1)) {
                *x = 0;
            } else if (non_finite<VT>(*x)) {
                *x = finite_only<VT>(*x);
                atomicMin(&bad[0], key0 + key);
                atomicMax(&bad[1], key0 + key);
            }
        });
    }
};

// Keeps what comes before it before what comes after it.  Left alone, the
// compiler puts each LDS read right before its use and gathers matrix
// instructions apart from the arithmetic that could run beside them.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// The operands of S^T: key lane % 32 of 32, 16 dims a step.
template <int DP>
struct KeyReads {
    using L = Tiles<DP>;
    const char *row;
    int piece;

    __device__ explicit KeyReads(const char *keys)
    {
        const int lane = int(threadIdx.x) & (kLanes - 1), col = lane & 31;
        piece = (lane >> 5) ^ L::key_swizzle(col);
        row = keys + col * L::kRow;
    }
    __device__ __forceinline__ u32x4 operator()(int step) const
    {
        return *reinterpret_cast<const u32x4 *>(row + ((piece ^ (2 * step)) << 4));
    }
};

// The operands of O^T, V^T: 32 dims of 16 keys a read (two of them).
template <int DP>
struct ValueReads {
    using L = Tiles<DP>;
    const char *from;
    int swizzle;

    __device__ explicit ValueReads(const char *values)
    {
        // lane i of 16 names key i / 4, four dims from 4 (i % 4), and gets dim i, keys 0-3
        const int lane = int(threadIdx.x) & (kLanes - 1);
        const int key = 4 * (lane >> 5) + (lane & 15) / 4;
        from = values + key * L::kRow + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
        swizzle = L::value_swizzle(key) >> 2;
    }
    __device__ __forceinline__ u32x4 operator()(int u, int dt) const       // keys 16 u ..., dims 32 dt ...
    {
        using Lds = __attribute__((address_space(3))) i16x4;
        const char *at = from + u * 16 * L::kRow + ((dt ^ swizzle) << 6);
        const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds *)at);
        const i16x4 z = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds *)(at + 8 * L::kRow));
        const u32x2 yy = __builtin_bit_cast(u32x2, y), zz = __builtin_bit_cast(u32x2, z);
        return u32x4{yy.x, yy.y, zz.x, zz.y};
    }
};

// The first operands of a tile, read before they are needed.
template <int DP> struct Ready {
    static constexpr int kN = Tiles<DP>::kDims < 4 ? Tiles<DP>::kDims : 4;
    u32x4 a[kN];
};

template <int DP>
__device__ __forceinline__ Ready<DP> read_ahead(const char *values)
{
    const ValueReads<DP> read(values);
    Ready<DP> r;
#pragma unroll
    for (int n = 0; n < Ready<DP>::kN; ++n) r.a[n] = read(0, n);
    return r;
}

// Hides what a row does not see: key j of the 32 is seen in [lo, hi) (relative
// to the first) if its 16-key group is there.
__device__ __forceinline__ void hide(f32x16 &s, int lo, int hi, uint32_t there)
{
    // register i holds key 8 (i / 4) + i % 4 + 4 half; the half goes to the
    // limits, so that the rest is a constant
    const int half = (int(threadIdx.x) & (kLanes - 1)) >> 5;
    lo -= 4 * half;
    hi -= 4 * half;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int key = 8 * (i / 4) + i % 4;
        const bool seen = key >= lo && key < hi && ((there >> (i / 8)) & 1);
        s[i] = seen ? s[i] : -INFINITY;
    }
}

// The larger of a column's two halves.
__device__ __forceinline__ float both_halves(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_elementwise_maximum(__builtin_bit_cast(float, uint32_t(r[0])),
                                         __builtin_bit_cast(float, uint32_t(r[1])));
}

// The exponent of a weight is (score - reference) c + lift.  Near zero (ONE) it
// takes one multiply-add, score * c less the reference times c: that product is
// rounded, up to kFar by at most 2^-13, which a weight shows as 1 in 10^4, no
// more than the scores' own rounding.  Further out it would be off by whole
// powers of two, and past 2^31 by all that fp32 holds: there the scores become
// differences to the reference first.  Where instructions are not what bounds a
// walk, or a second path costs it registers, every weight takes the difference
// (64 single tokens of up to 8192 keys 249 us with ONE, 244 without; the last
// 1024 tokens of 2 x 4096, 16 heads of 256 on 4, bf16 297 and 240, e4m3 371 and
// 379).
constexpr float kFar = 4096.0f;

// Takes the largest of a lane's scores s into the running maximum.  The
// reference moves only when a weight would pass 2^8: any reference within that
// of the true maximum gives the same softmax, and most tiles then leave O as
// it is, and ask no other lane.  With ONE and a reference past kFar in the
// wave, no score is below the limit and every tile comes here.
template <int VT, int DP, bool ONE>
__device__ __forceinline__ void move_top(Rows<DP> &r, f32x16 &s, float top, float c)
{
    if (__builtin_expect(__any(top > r.limit), 0)) {
        const float now = fmaxf(r.top, both_halves(top));
        const float keep = r.top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((r.top - now) * c);
        const float from = now == -INFINITY ? 0.0f : now;
        r.top = now;
        r.base = ONE ? fmaf(from, c, -lift<VT>()) : from;
        r.limit = now + 8.0f / c;
        if constexpr (ONE) {
            if (__builtin_expect(__any(fabsf(r.base) > kFar), 0)) {
                r.base = -lift<VT>();
                r.limit = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] -= from;
            }
        }
        r.sum *= keep;
#pragma unroll
        for (int dt = 0; dt < Tiles<DP>::kDims; ++dt) {
            r.o[dt] *= keep;
            in_order();
        }
    }
}

// Scores [from, to) of 32 keys to weights, added to sum; pairs are rounded to
// VT once both are there.
template <int VT, bool ONE>
__device__ __forceinline__ void exponentials(f32x16 &s, u32x4 (&w)[2], float &sum, float c, float base,
                                             int from, int to)
{
    typedef typename Elem<VT>::type V2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int n = from; n < to; ++n) {
        const float x = __builtin_amdgcn_exp2f(ONE ? fmaf(s[n], c, -base) : fmaf(s[n] - base, c, lift<VT>()));
        s[n] = x;
        sum += x;
        if (n % 2) {
            const f32x2 pair = {s[n - 1], x};
            uint32_t both = __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, V2));
            // here, and not where it is used: the compiler would otherwise sink
            // all of this past the branch that follows the matrix instructions
            asm volatile("" : "+v"(both), "+v"(sum));
            w[n / 8][n / 2 % 4] = both;
        }
    }
}

// No loads beside a run of matrix instructions.
struct NoLoads {
    __device__ __forceinline__ void operator()(int, int) const {}
};

// S^T of 32 keys.  The matrix instructions run beside the exponentials of the
// 32 keys before (BESIDE): a wave issues one and goes on, and 16 scores take
// about as long as the head's instructions do; loads(n, kN) issues what is to be
// issued beside the n-th of kN.
template <int DT, int VT, int DP, bool BESIDE, bool ONE, typename Loads>
__device__ __forceinline__ void scores(f32x16 &out, const u32x4 (&q)[Tiles<DP>::kSteps],
                                       const char *keys, f32x16 &s, u32x4 (&w)[2], float &sum, float c,
                                       float base, Loads loads)
{
    constexpr int kN = Tiles<DP>::kSteps, kAhead = kN < 4 ? kN : 4;
    const KeyReads<DP> read(keys);
    u32x4 a[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) a[n] = read(n);
    in_order();
    f32x16 o = 0.0f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        o = mfma<DT>(a[n % kAhead], q[n], o);
        if (n + kAhead < kN) a[n % kAhead] = read(n + kAhead);
        if constexpr (BESIDE) exponentials<VT, ONE>(s, w, sum, c, base, n * 16 / kN, (n + 1) * 16 / kN);
        loads(n, kN);
        in_order();
    }
    out = o;
}

// The largest of a lane's scores; NaN if one is (its row's sum is then NaN
// whatever the reference).  Three operands an instruction, and unlike fmaxf no
// extra one to quiet each score.
__device__ __forceinline__ float larger(float top, const f32x16 &s, int n)
{
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(s[n], s[n + 1]), top);
}

__device__ __forceinline__ float largest(const f32x16 &s)
{
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < 16; n += 2) top = larger(top, s, n);
    return top;
}

// O^T += V^T P^T for 32 keys; the largest of the next scores is found beside
// it (BESIDE).
template <int VT, int DP, bool BESIDE, typename Loads>
__device__ __forceinline__ void add_values(Rows<DP> &r, const u32x4 (&w)[2], const char *values,
                                           Ready<DP> ready, const f32x16 &next, float &top, Loads loads)
{
    constexpr int kDims = Tiles<DP>::kDims, kN = 2 * kDims, kAhead = Ready<DP>::kN;
    const ValueReads<DP> read(values);
    if constexpr (BESIDE) top = -INFINITY;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        r.o[n % kDims] = mfma<VT>(ready.a[n % kAhead], w[n / kDims], r.o[n % kDims]);
        const int m = n + kAhead;
        if (m < kN) ready.a[n % kAhead] = read(m / kDims, m % kDims);
        if constexpr (BESIDE) {
#pragma unroll
            for (int i = n * 8 / kN; i < (n + 1) * 8 / kN; ++i) top = larger(top, next, 2 * i);
        }
        loads(n, kN);
        in_order();
    }
}

// The infinities and NaN of four dims among the values that a row sees, added
// up (0 if there are none): any weight times one of them is it.  Keys in
// [lo, hi) that are on a page: those between the first and the last such value
// that was taken out (over all keys of a block, one infinity in the last place
// made 4096 tokens over 12288 keys take 62 ms instead of 0.7).
template <int CDT>
__device__ f32x4 non_finite_sum(const AttnParams &p, const int32_t *table, int kv_head, int d,
                                int lo, int hi)
{
    using C = typename Elem<CDT>::type;
    const PagedParams &g = p.paged;
    f32x4 sum = 0.0f;
    for (int key = lo; key < hi; ++key) {
        const int at = table[key >> g.page_shift];
        if (at < 0 || at >= g.n_pages) continue;
        const int64_t row = ((int64_t(at) * p.n_k_heads + kv_head) << g.page_shift) +
                            (key & ((1 << g.page_shift) - 1));
        const C *e = static_cast<const C *>(g.v_cache) + row * p.head_dim + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x;
            if constexpr (CDT == kE4M3) x = __builtin_amdgcn_cvt_f32_fp8(int(e[i]), 0);
            else x = float(e[i]);
            if (!__builtin_isfinite(x)) sum[i] += x;
        }
    }
    return sum;
}

template <int DT>
__device__ __forceinline__ void store4(typename Elem<DT>::type *p, f32x4 v)
{
    typedef typename Elem<DT>::type T4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<T4 *>(p) = __builtin_convertvector(v, T4);
}

struct Parts {
    float2 *stats;        // [splits][rows]: maximum, sum of weights
    float *o;             // [splits][rows][head_dim]
    int64_t rows;         // n_tokens * n_q_heads
};

template <int N> using Const = std::integral_constant<int, N>;

// The keys [from, to) of a tile by waves that own 32 rows each and share the
// keys in WAYS ways: way y takes keys from + 64 (WAYS t + y) in turn t.
//
// A turn is 64 keys in two halves.  While a wave turns the scores of 32 keys
// into weights, the matrix cores compute the scores of the next 32; while they
// add its values, it finds the next maximum.  Keys are therefore wanted half a
// turn before their values, and the key tiles in LDS lie half a turn ahead.
// Two buffers each; a turn's reads run for the whole turn before it.
template <int DT, int CDT, int DP, bool EXACT, int WAYS>
struct RowWalk {
    using L = Tiles<DP>;
    static constexpr int VT = Types<DT, CDT>::V, kWaves = L::kWaves / WAYS;
    static constexpr int kHalf = 32 * L::kRow, kTile = 2 * kHalf, kStride = 64 * WAYS;
    static constexpr bool kOne = DP <= 128 || CDT == kE4M3;          // of move_top
    using Keys = Stage<DT, CDT, DP, EXACT, kWaves, true>;
    using Vals = Stage<DT, CDT, DP, EXACT, kWaves, false>;

    const AttnParams &p;
    const Plan &w;
    const int from, to, first;
    char *lds;
    const uint32_t at;
    Keys sk;                          // its tile t + 1: what follows the first half of turn t
    Vals sv;

    __device__ RowWalk(const AttnParams &p, const Plan &w, int kv_head, int wave, int from, int to, char *lds)
        : p(p), w(w), from(from), to(to), first(from + wave / kWaves * 64),
          lds(lds + wave / kWaves * 4 * kTile), at(lds_address(this->lds)),
          sk(p, w, kv_head, wave % kWaves, first - kStride, kStride, from, to),
          sv(p, w, kv_head, wave % kWaves, first, kStride, from, to)
    {
        sk.find_pages(0);
        sv.find_pages(0);
        sk.template fetch<false>(0, at);
    }

    // lo, hi: the limits of this lane's row.
    __device__ __forceinline__ void run(int group, int lo, int hi, float c,
                                        const u32x4 (&q)[Tiles<DP>::kSteps], int *bad, Rows<DP> &r)
    {
        // limits of all of the wave's rows (they grow with the row), and of the tile's
        const int wave_hi = min(__builtin_amdgcn_readlane(hi, 31), to);
        const int plain_lo = __builtin_amdgcn_readlane(lo, 31);
        const int plain_hi = min(__builtin_amdgcn_readlane(hi, 0), to) - 32;
        // keys that every row of the tile sees; elsewhere values are looked at
        int blo, bhi, unused;
        row_limits(p, w, w.row0 + w.rows - 1, group, blo, unused);
        row_limits(p, w, w.row0, group, unused, bhi);
        bhi = min(bhi, to);
        hi = min(hi, to);

        const int n_turns = (to - from + kStride - 1) / kStride;
        const auto part_hidden = [&](int key0, uint32_t there) {
            return key0 < plain_lo || key0 > plain_hi || (there & 3) != 3;
        };

        f32x16 a, b;                          // scores of a turn's halves
        u32x4 x[2];
        float top, none = 0.0f;
        uint32_t there = 0, next_there = sv.groups_there(0);   // groups on a page, of this turn and the next
        // Begins turn t: its keys and values are there, every wave is done
        // with the last turn's buffers, and the next turn's values and the
        // keys after them may be read.  The last turn reads what nobody wants,
        // from page 0.
        const char *next_keys, *next_values;
        uint32_t keys_at, values_at;
        const auto begin = [&](int t, char *keys, char *values) {
            if constexpr (Keys::kDirect) {
                wait_loads<0>();
            } else {
                sk.template store<false>(keys);
                if (t >= 0) sv.template store<true>(values);
            }
            const int key0 = first + t * kStride;
            if (t >= 0 && (key0 < blo || key0 + 64 > bhi || there != 15))
                sv.clean_values(values, t, there, bad);
            __syncthreads();
            if ((t + 1) % Vals::kBatch == 0 && t >= 0) sv.find_pages(t + 1);
            if ((t + 2) % Keys::kBatch == 0) sk.find_pages(t + 2);
            next_there = sv.groups_there(t + 1);
            next_values = sv.group_at(p.paged.v_cache, t + 1, 0);
            next_keys = sk.group_at(p.paged.k_cache, t + 2, 0);
            keys_at = at + (t & 1) * kTile;
            values_at = at + (2 + ((t + 1) & 1)) * kTile;
        };
        const auto load = [&](int i) {        // of 2 kSlots
            if (i % 2 == 0) sv.template fetch_part<true>(next_values, 0, i / 2, values_at);
            else sk.template fetch_part<false>(next_keys, 0, i / 2, keys_at);
        };
        // The loads are spread over a turn: a CU's address unit takes 16
        // cycles for each, and a wave that meets it busy waits.
        const auto quarter = [&](auto which) {
            return [&](int n, int of) {
                constexpr int kLo = decltype(which)::value * 2 * Vals::kSlots / 4;
                constexpr int kHi = (decltype(which)::value + 1) * 2 * Vals::kSlots / 4;
#pragma unroll
                for (int i = kLo; i < kHi; ++i)
                    if ((i - kLo) * of / (kHi > kLo ? kHi - kLo : 1) == n) load(i);
            };
        };
        const auto all_loads = [&] {
#pragma unroll
            for (int i = 0; i < 2 * Vals::kSlots; ++i) load(i);
        };

        begin(-1, lds, lds);                  // brings the first 32 keys
        all_loads();
        scores<DT, VT, DP, false, kOne>(a, q, lds + kHalf, b, x, none, c, 0.0f, NoLoads{});
        hide(a, lo - first, hi - first, next_there);
        top = largest(a);
        for (int t = 0; t < n_turns; ++t) {
            char *keys = lds + ((t + 1) & 1) * kTile, *values = lds + (2 + (t & 1)) * kTile;
            const int key0 = first + t * kStride;
            there = next_there;
            begin(t, keys, values);
            if (key0 >= wave_hi) {            // past what the wave's rows see
                all_loads();
                continue;
            }
            const bool hide_b = part_hidden(key0 + 32, there >> 2);
            const bool hide_a = part_hidden(key0 + kStride, next_there);
            move_top<VT, DP, kOne>(r, a, top, c);
            scores<DT, VT, DP, true, kOne>(b, q, keys, a, x, r.sum, c, r.base, quarter(Const<0>{}));
            Ready<DP> ready = read_ahead<DP>(values);
            if (hide_b) hide(b, lo - key0 - 32, hi - key0 - 32, there >> 2);
            in_order();
            add_values<VT, DP, true>(r, x, values, ready, b, top, quarter(Const<1>{}));
            move_top<VT, DP, kOne>(r, b, top, c);
            // in the last turn the next scores are of keys that nobody wants,
            // and so is their maximum
            scores<DT, VT, DP, true, kOne>(a, q, keys + kHalf, b, x, r.sum, c, r.base, quarter(Const<2>{}));
            ready = read_ahead<DP>(values + kHalf);
            if (hide_a) hide(a, lo - key0 - kStride, hi - key0 - kStride, next_there);
            in_order();
            add_values<VT, DP, true>(r, x, values + kHalf, ready, a, top, quarter(Const<3>{}));
        }
        wait_loads<0>();                      // before anyone else uses the buffers
    }
};

// The keys [from, to) of a tile whose rows every wave has: a wave takes every
// kWaves-th 32 keys.  It has a buffer of its own: the next keys are read once
// the scores are done with these, the next values once O is.
template <int DT, int CDT, int DP, bool EXACT>
struct KeyWalk {
    using L = Tiles<DP>;
    using S = Stage<DT, CDT, DP, EXACT, 1, false>;
    static constexpr int VT = Types<DT, CDT>::V;
    static constexpr int kStep = 32 * L::kWaves, kHalf = 32 * L::kRow;

    const int to, first, n_tiles;
    char *keys;
    const uint32_t at;
    S st;

    __device__ KeyWalk(const AttnParams &p, const Plan &w, int kv_head, int wave, int from, int to, char *lds)
        : to(to), first(from + wave * 32), n_tiles(to > first ? (to - first + kStep - 1) / kStep : 0),
          keys(lds + wave * 2 * kHalf), at(lds_address(keys)), st(p, w, kv_head, 0, first, kStep, from, to)
    {
        if (n_tiles == 0) return;
        st.find_pages(0);
        st.template fetch<false>(0, at);
        st.template fetch<true>(0, at + kHalf);
    }

    __device__ __forceinline__ void run(int lo, int hi, float c, const u32x4 (&q)[Tiles<DP>::kSteps],
                                        int *bad, Rows<DP> &r)
    {
        char *values = keys + kHalf;
        hi = min(hi, to);
        const int plain_lo = __builtin_amdgcn_readlane(lo, 31);
        const int plain_hi = __builtin_amdgcn_readlane(hi, 0) - 32;
        for (int t = 0; t < n_tiles; ++t) {
            const int key0 = first + t * kStep;
            const bool more = t + 1 < n_tiles;
            const uint32_t there = st.groups_there(t);
            f32x16 s;
            u32x4 x[2];
            float unused;
            if constexpr (S::kDirect) {
                wait_loads<S::kLoads>();             // the values may be on their way
            } else {
                st.template store<false>(keys);
                st.template store<true>(values);
            }
            scores<DT, VT, DP, false, false>(s, q, keys, s, x, r.sum, c, 0.0f, NoLoads{});
            if (more) {
                if ((t + 1) % S::kBatch == 0) st.find_pages(t + 1);
                wait_lds();
                st.template fetch<false>(t + 1, at);
                if constexpr (!S::kDirect) st.template fetch<true>(t + 1, at + kHalf);
            }
            const bool whole = key0 >= plain_lo && key0 <= plain_hi && there == 3;
            if (!whole) hide(s, lo - key0, hi - key0, there);
            move_top<VT, DP, false>(r, s, largest(s), c);
            exponentials<VT, false>(s, x, r.sum, c, r.base, 0, 16);
            if constexpr (S::kDirect) {
                if (more) wait_loads<S::kLoads>();
                else wait_loads<0>();
            }
            if (!whole) st.clean_values(values, t, there, bad);
            add_values<VT, DP, false>(r, x, values, read_ahead<DP>(values), s, unused, NoLoads{});
            if constexpr (S::kDirect) {
                wait_lds();
                if (more) st.template fetch<true>(t + 1, at + kHalf);
            }
        }
    }
};

template <int DT, int CDT, int DP, bool EXACT>
__global__ __launch_bounds__(Tiles<DP>::kWaves *kLanes, DP > 128 ? 1 : 2) void attend(
    AttnParams p, Parts parts, int tiles, int tile_rows, int max_splits)
{
    using T = typename Elem<DT>::type;
    using L = Tiles<DP>;
    constexpr int kWaves = L::kWaves;
    __shared__ __attribute__((aligned(16))) char lds[L::kLds];
    __shared__ int bad[2];       // keys between which values that are not finite were taken out
    __shared__ float wave_stats[kWaves][32][2];
    __shared__ int64_t wave_rows[kWaves][32][2];

    const PagedParams &g = p.paged;
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kLanes);
    const int col = lane & 31, half = lane >> 5;
    const int group = p.n_q_heads / p.n_k_heads;
    // heads vary fastest: blocks go to the XCDs in turn, so that with eight
    // key heads each XCD's L2 serves one; long tiles (late rows) start first
    const int kv_head = int(blockIdx.x) % p.n_k_heads;
    const int tile = tiles - 1 - int(blockIdx.x) / p.n_k_heads;
    const int split = int(blockIdx.y);

    Plan w;
    if (!find_tile(p, w, tile, group, tile_rows)) return;
    plan_keys(p, w, group, tile_rows, max_splits);
    if (split >= w.splits) return;
    const int from = w.lo + split * w.per;
    const int to = min(w.hi, from + w.per);
    // waves that share their rows: all, two and two, or none
    const int ways = w.rows <= kRowsPerWave ? kWaves
                     : (kWaves == 8 && w.rows <= 4 * kRowsPerWave ? 2 : 1);
    const int row_waves = kWaves / ways;

    // this lane's row and its limits (rows past the last repeat it)
    const int first = wave % row_waves * kRowsPerWave;
    const int row = w.row0 + min(first + col, w.rows - 1);
    const int token = w.begin + row / group, head = kv_head * group + row % group;
    int lo, hi;
    row_limits(p, w, row, group, lo, hi);
    const T *src = static_cast<const T *>(p.q) + int64_t(token) * p.q_stride +
                   int64_t(head) * p.head_dim + half * 8;
    // its place among the outputs, for the way out
    if (half == 0) {
        wave_rows[wave][col][0] = int64_t(token) * p.out_stride + int64_t(head) * p.head_dim;
        wave_rows[wave][col][1] = split * parts.rows + int64_t(token) * p.n_q_heads + head;
    }
    const float c = p.scale * g.k_scale * kLog2e;
    if (threadIdx.x < 2) bad[threadIdx.x] = threadIdx.x == 0 ? INT32_MAX : -1;
    __syncthreads();

    u32x4 q[L::kSteps];
    const auto read_queries = [&] {
#pragma unroll
        for (int st = 0; st < L::kSteps; ++st)
            q[st] = EXACT || st * 16 < p.head_dim ? *reinterpret_cast<const u32x4 *>(src + st * 16) : u32x4(0u);
        // wait for them here: a wait inside the loop would be one for the next
        // tile's reads as well.  Wide heads of e4m3 caches, whose keys and
        // values pass through registers, leave these no other place than the
        // accumulators' side (with addresses made at each load: 766 -> 427 us for 2 x 1024
        // tokens over 4096 keys, 16 heads on 4)
#pragma unroll
        for (int st = 0; st < L::kSteps; ++st) {
            if constexpr (DP > 128 && CDT == kE4M3) asm volatile("" : "+a"(q[st]));
            else asm volatile("" : "+v"(q[st]));
        }
    };
    Rows<DP> r;
    // each walk begins its first reads when it is made; the queries come beside them
    if (ways == 1) {
        RowWalk<DT, CDT, DP, EXACT, 1> walk(p, w, kv_head, wave, from, to, lds);
        read_queries();
        walk.run(group, lo, hi, c, q, bad, r);
    } else if (ways == 2) {
        RowWalk<DT, CDT, DP, EXACT, kWaves == 8 ? 2 : 1> walk(p, w, kv_head, wave, from, to, lds);
        read_queries();
        walk.run(group, lo, hi, c, q, bad, r);
    } else {
        KeyWalk<DT, CDT, DP, EXACT> walk(p, w, kv_head, wave, from, to, lds);
        read_queries();
        walk.run(lo, hi, c, q, bad, r);
    }
    r.sum += __shfl_xor(r.sum, 32);

    // Every wave's O goes through LDS, so that stores are whole rows; waves
    // with the same rows bring theirs to a common maximum and are added.
    if (half == 0) {
        wave_stats[wave][col][0] = r.top;
        wave_stats[wave][col][1] = r.sum;
    }
    __syncthreads();
    const auto weight = [&](float t, float top) {
        return t == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((t - top) * c);
    };
    constexpr int kRow = L::kSumRow;
    float *all = reinterpret_cast<float *>(lds);      // [wave][row][kRow]
    if (first + col < w.rows) {
        float keep = 1.0f;
        if (ways > 1) {
            float top = r.top;
            for (int i = wave % row_waves; i < kWaves; i += row_waves) top = fmaxf(top, wave_stats[i][col][0]);
            keep = weight(r.top, top);
        }
#pragma unroll
        for (int dt = 0; dt < L::kDims; ++dt)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int d = dt * 32 + 8 * b + 4 * half;
                if (d >= DP) continue;
                f32x4 x = {r.o[dt][4 * b], r.o[dt][4 * b + 1], r.o[dt][4 * b + 2], r.o[dt][4 * b + 3]};
                *reinterpret_cast<f32x4 *>(all + (wave * 32 + col) * kRow + d) = x * keep;
            }
    }
    __syncthreads();
    // four dims a lane, a row to 32 or 64 lanes
    constexpr int kRowLanes = DP <= 128 ? 32 : 64, kRowsAtOnce = kWaves * kLanes / kRowLanes;
    const int d = int(threadIdx.x) % kRowLanes * 4;
    const int bad_lo = bad[0], bad_hi = bad[1] + 1;
    for (int n = int(threadIdx.x) / kRowLanes; n < w.rows; n += kRowsAtOnce) {
        if (d >= p.head_dim) continue;
        const int k0 = n / 32, col = n % 32;
        f32x4 x = *reinterpret_cast<const f32x4 *>(all + n * kRow + d);
        float top = wave_stats[k0][col][0], sum = wave_stats[k0][col][1];
        if (ways > 1) {
            const float own = top;
            for (int k = k0 + row_waves; k < kWaves; k += row_waves) {
                x += *reinterpret_cast<const f32x4 *>(all + (k * 32 + col) * kRow + d);
                top = fmaxf(top, wave_stats[k][col][0]);
            }
            sum = sum == 0.0f ? 0.0f : sum * weight(own, top);
            for (int k = k0 + row_waves; k < kWaves; k += row_waves) {
                const float part = wave_stats[k][col][1];
                if (part != 0.0f) sum += part * weight(wave_stats[k][col][0], top);
            }
        }
        if (bad_lo < bad_hi) {
            int lo, hi;
            row_limits(p, w, w.row0 + n, group, lo, hi);
            x += non_finite_sum<CDT>(p, g.block_table + int64_t(w.seq) * g.max_pages, kv_head, d,
                                     max(lo, bad_lo), min(hi, bad_hi));
        }
        if (w.splits == 1) {
            x *= sum == 0.0f ? 0.0f : g.v_scale / sum;
            store4<DT>(static_cast<T *>(p.out) + wave_rows[k0][col][0] + d, x);
        } else {
            const int64_t part = wave_rows[k0][col][1];
            *reinterpret_cast<f32x4 *>(parts.o + part * p.head_dim + d) = x;
            if (d == 0) parts.stats[part] = make_float2(top, sum);
        }
    }
}

// Adds the splits of the rows of a tile; tiles of one split are already in
// place.  The rows of a tile go to gridDim.y blocks in turn; a thread takes
// four dims of a row, or, where a block has few rows, `ways` threads share the
// splits and meet in LDS.
constexpr int kJoinBlock = 512;

struct Sum {
    float top, sum;      // maximum, sum of weights
    f32x4 o;
};

__device__ __forceinline__ float part_weight(float top, float all, float c)
{
    // scores that are all NaN leave no maximum, but a sum
    return top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((top - all) * c);
}

template <int DT>
__global__ __launch_bounds__(kJoinBlock) void attend_join(AttnParams p, Parts parts, int tile_rows,
                                                          int max_splits)
{
    using T = typename Elem<DT>::type;
    __shared__ Sum shared[kJoinBlock];
    const int group = p.n_q_heads / p.n_k_heads;
    const int kv_head = int(blockIdx.x) % p.n_k_heads;
    Plan w;
    if (!find_tile(p, w, int(blockIdx.x) / p.n_k_heads, group, tile_rows)) return;
    plan_keys(p, w, group, tile_rows, max_splits);
    if (w.splits == 1) return;

    const float c = p.scale * p.paged.k_scale * kLog2e;
    const int turn = int(gridDim.y), rows = (w.rows - int(blockIdx.y) + turn - 1) / turn;
    const int fours = p.head_dim / 4, n = rows * fours;
    int ways = 1;
    while (ways * 2 * n <= kJoinBlock && ways < w.splits) ways *= 2;
    const int per_way = kJoinBlock / ways;
    const int way = int(threadIdx.x) / per_way;

    const auto row_of = [&](int i) { return w.row0 + int(blockIdx.y) + i / fours * turn; };
    const auto put = [&](int row, int d, const Sum &a) {
        const float f = a.sum == 0.0f ? 0.0f : p.paged.v_scale / a.sum;
        store4<DT>(static_cast<T *>(p.out) + int64_t(w.begin + row / group) * p.out_stride +
                       int64_t(kv_head * group + row % group) * p.head_dim + d, a.o * f);
    };
    for (int i = int(threadIdx.x) % per_way; i < n; i += per_way) {
        const int row = row_of(i), d = i % fours * 4;
        const int64_t at = int64_t(w.begin + row / group) * p.n_q_heads + kv_head * group + row % group;
        const float2 *stats = parts.stats + at;
        const float *o = parts.o + at * p.head_dim + d;
        Sum a = {-INFINITY, 0.0f, f32x4(0.0f)};
#pragma unroll 4
        for (int k = way; k < w.splits; k += ways) a.top = fmaxf(a.top, stats[k * parts.rows].x);
#pragma unroll 4
        for (int k = way; k < w.splits; k += ways) {
            const float2 st = stats[k * parts.rows];
            const f32x4 x = *reinterpret_cast<const f32x4 *>(o + k * parts.rows * p.head_dim);
            const float f = st.y == 0.0f ? 0.0f : part_weight(st.x, a.top, c);   // 0: saw no key
            a.sum += st.y * f;
            a.o += x * f;
        }
        if (ways > 1) shared[threadIdx.x] = a;     // n <= per_way: the only turn of the loop
        else put(row, d, a);
    }
    if (ways == 1) return;
    __syncthreads();
    const int i = int(threadIdx.x);
    if (i >= n) return;
    Sum a = {-INFINITY, 0.0f, f32x4(0.0f)};
    for (int k = 0; k < ways; ++k) a.top = fmaxf(a.top, shared[k * per_way + i].top);
    for (int k = 0; k < ways; ++k) {
        const Sum &b = shared[k * per_way + i];
        const float f = b.sum == 0.0f ? 0.0f : part_weight(b.top, a.top, c);
        a.sum += b.sum * f;
        a.o += b.o * f;
    }
    put(row_of(i), i % fours * 4, a);
}

// Parts of the launch: rows of a tile, tiles (an upper bound that needs no
// look at the offsets) and splits of the keys.
struct Shape { int tile_rows; int64_t tiles; int splits; };

Shape shape_of(int64_t n_tokens, int32_t n_seqs, int32_t n_q_heads, int32_t n_k_heads,
               int32_t head_dim, int32_t page_size, int32_t max_pages)
{
    const int64_t group = n_q_heads / n_k_heads, rows = n_tokens * group;
    const int64_t slots = 256;           // blocks the chip holds: one for each CU
    const int64_t units = (int64_t(max_pages) * page_size + kUnit - 1) / kUnit;
    Shape s = {128, rows / 128 + n_seqs, 1};
    if (rows <= int64_t(n_seqs) * kRowsPerWave) {
        // Few rows: the keys are read once and HBM decides, so the chip is
        // filled once.  Two sequences of 131072 keys, 4 heads, e4m3: 32 splits
        // 54 us, 16 66, 64 60, 128 73.  A join costs as much as 8 units: one
        // sequence, 8 heads, of 2048 keys 13.3 us whole and 13.8 split, of
        // 4096 24 and 16.
        const int64_t blocks = s.tiles * n_k_heads;
        if (blocks == 0 || units <= 8) return s;
        const int64_t n = slots / blocks < units ? slots / blocks : units;
        s.splits = int(n < 1 ? 1 : n);
        return s;
    }
    // Many rows: the blocks run in rounds of `slots`.  In units' times of 128
    // rows, a block takes one or (256 rows, no waves that share keys) two for
    // each unit, 6 or 8 to begin and end, and the join one and more with its
    // splits.  Tiles of 128 rows
    // against 256: 288 blocks of 2816 keys 90 us and 78, 1024 of up to 12288
    // 755 and 710, 228 of up to 6333 74 and 104 (the rule takes the better in
    // each); 16 blocks of 8192 keys 131 us whole and 37 in 16 splits; one of
    // 131072 keys (a token of 64 heads on one) 137 in 16 and 63 in up to 64.
    int64_t best = INT64_MAX;
    for (int tile_rows = 128; tile_rows <= (head_dim <= 128 ? 256 : 128); tile_rows *= 2) {
        const int64_t full = (rows + int64_t(n_seqs - 1) * (tile_rows / 2) + tile_rows - 1) / tile_rows *
                             n_k_heads;                    // about the tiles that have rows
        for (int n = 1; n <= 64 && n <= units; ++n) {
            const int64_t block = (units + n - 1) / n * (tile_rows / 128) + 4 + tile_rows / 64;
            const int64_t cost = (full * n + slots - 1) / slots * block + (n > 1 ? 1 + n / 16 : 0);
            if (cost >= best) continue;
            best = cost;
            s = {tile_rows, rows / tile_rows + n_seqs, n};
        }
    }
    return s;
}

size_t round_up(size_t n) { return (n + 255) & ~size_t(255); }

template <int DT, int CDT, int DP, bool EXACT>
void launch(const AttnParams &p, const Parts &parts, const Shape &s, hipStream_t stream)
{
    const dim3 grid(uint32_t(s.tiles * p.n_k_heads), uint32_t(s.splits));
    attend<DT, CDT, DP, EXACT><<<grid, Tiles<DP>::kWaves * kLanes, 0, stream>>>(
        p, parts, int(s.tiles), s.tile_rows, s.splits);
}

// Common widths have kernels of their own; the others take the next of three,
// with zeros behind the head.
template <int DT, int CDT>
void launch_attend(const AttnParams &p, const Parts &parts, const Shape &s, hipStream_t stream)
{
    const int d = p.head_dim;
    if (d == 64) launch<DT, CDT, 64, true>(p, parts, s, stream);
    else if (d == 80) launch<DT, CDT, 80, true>(p, parts, s, stream);
    else if (d == 96) launch<DT, CDT, 96, true>(p, parts, s, stream);
    else if (d == 128) launch<DT, CDT, 128, true>(p, parts, s, stream);
    else if (d == 256) launch<DT, CDT, 256, true>(p, parts, s, stream);
    else if (d < 64) launch<DT, CDT, 64, false>(p, parts, s, stream);
    else if (d < 128) launch<DT, CDT, 128, false>(p, parts, s, stream);
    else launch<DT, CDT, 256, false>(p, parts, s, stream);
}

}  // namespace

size_t attention_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t n_q_heads,
                                 int32_t n_k_heads, int32_t head_dim, int32_t page_size,
                                 int32_t max_pages)
{
    const Shape s = shape_of(n_tokens, n_seqs, n_q_heads, n_k_heads, head_dim, page_size,
                             max_pages);
    if (s.splits == 1) return 256;
    const size_t rows = size_t(n_tokens) * n_q_heads;
    return round_up(s.splits * rows * sizeof(float2)) + s.splits * rows * head_dim * sizeof(float);
}

hipError_t run_paged_attention(const AttnParams &p, hipStream_t stream)
{
    const Shape s = shape_of(p.n_tokens, p.paged.n_seqs, p.n_q_heads, p.n_k_heads, p.head_dim,
                             1 << p.paged.page_shift, p.paged.max_pages);
    Parts parts;
    parts.rows = int64_t(p.n_tokens) * p.n_q_heads;
    parts.stats = static_cast<float2 *>(p.workspace);
    parts.o = reinterpret_cast<float *>(static_cast<char *>(p.workspace) +
                                        round_up(s.splits * parts.rows * sizeof(float2)));
    const bool e4m3 = p.paged.cache_dtype == kE4M3;
    if (p.dtype == kF16 && !e4m3) launch_attend<kF16, kF16>(p, parts, s, stream);
    else if (p.dtype == kF16) launch_attend<kF16, kE4M3>(p, parts, s, stream);
    else if (!e4m3) launch_attend<kBF16, kBF16>(p, parts, s, stream);
    else launch_attend<kBF16, kE4M3>(p, parts, s, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.splits == 1) return e;
    // 16 rows a block; tiles of few rows and few splits are done by one (320
    // tiles, 2 splits: 241 us against 249)
    const bool few = parts.rows <= int64_t(p.paged.n_seqs) * p.n_k_heads * kRowsPerWave;
    const dim3 blocks(uint32_t(s.tiles * p.n_k_heads),
                      few && s.splits < 16 ? 1 : uint32_t(s.tile_rows / 16));
    if (p.dtype == kF16) attend_join<kF16><<<blocks, kJoinBlock, 0, stream>>>(p, parts, s.tile_rows, s.splits);
    else attend_join<kBF16><<<blocks, kJoinBlock, 0, stream>>>(p, parts, s.tile_rows, s.splits);
    return hipGetLastError();
}

}  // namespace bevpool
