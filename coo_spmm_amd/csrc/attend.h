// attend.h -- attention over the 8- and 4-bit cache: the kernel that streams it.
//
//   s_t = scale q . k_t,  out = sum_t softmax(s)_t v_t over the tokens a query sees
//
// One pass over the cache with a running maximum and sum.  Up to 16 queries of one
// cache head (a sequence's newest tokens times the query heads that share it) are
// the columns of both matrix products, S^T = K Q^T and O^T = V^T P^T (16x16x32,
// bf16): each lane then holds one query throughout, its scores' maximum, sum and
// rescaling are its own, and its probabilities are at once the second product's
// operand.  Codes go from memory straight into operand registers (cache.h has the
// layout); a cached value is a bf16 number (steps of 2^-133).  An fp32 query is split into
// three bf16 numbers whose sum it is, and so is every probability: three exact
// products added in fp32, for which there is room, since the cache's bytes bound
// this kernel.  With bf16 queries the probabilities keep 16 bits (two numbers).
//
// Work is cut without regard to the sequences' ends: all (sequence, queries, head)
// units one after the other are a row of tiles, of which every workgroup takes an
// equal run, its four wavefronts taking tiles in turn.  So one long sequence among
// short ones fills the card like any other batch.  A unit that one workgroup has
// whole is written by it; the pieces of the others are joined by a second launch in
// a fixed order.
//
// Measured (both launches): 64 streams of 256 to 4096 tokens, 8 cache heads of 128 in
// 4 bits, 154 MB, fp32 queries 49 us; one of 131072 tokens, 143 MB, bf16 queries 37 us
// (a copy's rate would be 30 and 28); 512 queries over 8192 tokens, int8, 67 GFLOP,
// bf16 (two products with V) 132 us; four prompts of 1024 tokens, 12 heads of 64, fp32
// (three products each) 55 us.
#pragma once

#include "cache.h"
#include "rope.h"

namespace snack {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttendWaves = 4;
constexpr int kAttendThreads = kAttendWaves * kWave;
constexpr int kQueries = 16;          // queries of a unit
constexpr int kAttendGroups = 512;   // workgroups at most: two a compute unit
// What a unit costs, in tiles.  Measured (us, both launches): blocks of 16 queries with 4 : 14 : 28, 64 streams of 256
// to 4096 tokens 51 : 47 : 52, 8 of 1000 17.5 : 15.6 : 15.8, one token over 16384 16.5 : 14.6 : 14.6; the others with
// 0 : 4 : 14, 512 queries over 8192 tokens 144 : 135 : 138, four prompts of 1024 64 : 56 : 66, 64 of 64 over 200
// 31 : 31 : 35.
constexpr int kFewCost = 14, kManyCost = 4;
constexpr int kMinRun = 4;            // tiles of a workgroup at least: one a wavefront
constexpr float kRaise = 8.0f;        // a running maximum is raised when a score passes it by a factor of 2^8

struct AttendArgs {
    const void* q;
    int64_t q_row, q_head;
    void* out;
    CacheView c;
    const int32_t* table;
    int32_t width, pages;
    const int32_t* lens;
    const int32_t* starts;
    int32_t sequences, per, tokens;   // per: tokens of a sequence where starts is null
    int32_t most_blocks;              // blocks of queries of a cache head that ascending starts can give
    int32_t hq;
    FastDiv by_group;                 // query heads of a cache head
    float scale_log2;                 // scale * log2(e)
    int32_t causal;
    float* part;                      // two partial results a workgroup: of the block it goes on with, of the one it starts
    // What the second launch reads, two to a workgroup or (by_unit) to a unit, a block of queries of one cache head, in
    // the order of the work: of a unit that a workgroup starts and does not end {sequence's first token, block, head,
    // pieces}, {its queries of a head, the workgroup, the last token that the sequence's first query sees}, else no
    // pieces.  The last: how many units there are.
    int4* meta;
    int32_t by_unit;
    int32_t meta_last;
};

// floats of a partial result of 16 queries: the output's, then maximum and sum of every query
__host__ __device__ constexpr int part_floats(int nb) { return 2 * nb * 256 + 2 * kQueries; }

// What nothing writes while the kernel runs, read by scalar loads where the address is the same for a wavefront (they
// do not queue behind the vector loads in flight).
template <typename T>
using Fixed = const __attribute__((address_space(4))) T*;
template <typename T>
__device__ inline Fixed<T> fixed(const T* p)
{
    return (Fixed<T>)(uintptr_t)p;
}

// a sequence of the call
struct Seq {
    int32_t first, nq, len;
    int32_t tiles;    // at least 1 (a query that sees nothing is still answered)
};
__device__ inline Seq get_seq(const AttendArgs& a, int32_t b)
{
    Seq s;
    int32_t last;
    if (a.starts) {
        s.first = min(max(fixed(a.starts)[b], 0), a.tokens);
        last = min(max(fixed(a.starts)[b + 1], s.first), a.tokens);
    } else {
        s.first = b * a.per;
        last = s.first + a.per;
    }
    s.nq = last - s.first;
    s.len = max(fixed(a.lens)[b], 0);
    // tokens past the page table are one more tile, which stands for all of them
    const int64_t room = (int64_t)a.width * a.c.page_tiles + 1;
    const int64_t t = ((int64_t)s.len + kTile - 1) / kTile;
    s.tiles = (int32_t)(t < 1 ? 1 : t < room ? t : room);
    return s;
}

// The queries of a cache head in a sequence (its tokens times the query heads of the group) are cut into blocks of
// ROWS.  A block takes its tiles up to the last one that its last query sees.
template <int ROWS>
__device__ inline int32_t seq_blocks(const AttendArgs& a, const Seq& s)
{
    return (int32_t)(((uint32_t)s.nq * a.by_group.d + ROWS - 1) / ROWS);
}
template <int ROWS>
__device__ inline int32_t block_tiles(const AttendArgs& a, const Seq& s, int32_t k)
{
    if (!a.causal) return s.tiles;
    const uint32_t rows = (uint32_t)s.nq * a.by_group.d, last = min((uint32_t)(k + 1) * ROWS, rows) - 1;
    const int64_t seen = (int64_t)s.len - s.nq + fast_quot(a.by_group, last) + 1;
    const int64_t t = (seen + kTile - 1) >> 5;
    return (int32_t)(t < 1 ? 1 : t < s.tiles ? t : s.tiles);
}

// The work: for every sequence, every block of queries, every cache head (a unit), what the unit itself costs, in tiles
// (queries to load, the first tiles to wait for, results to write), then its tiles, all one after the other.  Without
// the former a workgroup that gets many short units ends long after the others (64 streams of 256 to 4096 tokens: 68
// against 47 us).  A position within the former belongs to no workgroup: the one that has the unit's first tile
// starts it.  Where a position of this row lies:
struct Cursor {
    int32_t b, k;             // sequence, block
    int32_t blocks, tiles;    // of the sequence, of the block (of every head of it)
    int32_t cost;             // positions of a unit
    Seq s;
};
template <int ROWS>
__host__ __device__ constexpr int unit_cost()
{
    return ROWS == kQueries ? kFewCost : kManyCost;
}
template <int ROWS>
__device__ inline void set_cursor(const AttendArgs& a, Cursor& c, int32_t b, int32_t k)
{
    c.b = b;
    c.k = k;
    c.s = get_seq(a, b);
    c.blocks = seq_blocks<ROWS>(a, c.s);
}
// the next block; past the last sequence c.b is the number of sequences
template <int ROWS>
__device__ inline void next_block(const AttendArgs& a, Cursor& c)
{
    ++c.k;
    while (c.k >= c.blocks) {
        if (c.b + 1 >= a.sequences) {
            c.b = a.sequences;
            return;
        }
        set_cursor<ROWS>(a, c, c.b + 1, 0);
    }
    c.tiles = block_tiles<ROWS>(a, c.s, c.k);
    c.cost = c.tiles + unit_cost<ROWS>();
}

// x's sum over the threads before this one; lds holds THREADS / 64 numbers more than it takes, of which the first
// THREADS get the sums
template <int THREADS, typename T>
__device__ inline T group_scan(T x, T* lds, T* total)
{
    const int lane = (int)threadIdx.x & (kWave - 1), wave = (int)threadIdx.x / kWave;
    T y = x;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const T z = __shfl_up(y, d, kWave);
        if (lane >= d) y += z;
    }
    if (lane == kWave - 1) lds[THREADS + wave] = y;
    __syncthreads();
    T sum = 0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) {
        if (i == wave) y += sum;
        sum += lds[THREADS + i];
    }
    lds[threadIdx.x] = y - x;
    __syncthreads();
    *total = sum;
    return y - x;
}
// the last of n ascending numbers that is at most x (the first is)
template <int N, typename T>
__device__ inline int last_at_most(const T* v, T x)
{
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (v[m] <= x) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// The workgroup's threads take a run of sequences each to count the blocks, then a run of blocks each to count the
// tiles.
template <int THREADS>
struct Schedule {
    int64_t seqs[THREADS + THREADS / kWave];   // blocks before a thread's run of sequences
    int64_t work[THREADS + THREADS / kWave];   // tiles before a thread's run of blocks
};
template <int THREADS, int ROWS>
__device__ inline Cursor find_block(const AttendArgs& a, const Schedule<THREADS>& l, int32_t i)
{
    Cursor c;
    if (!a.starts) {
        const int32_t blocks = (int32_t)(((uint32_t)a.per * a.by_group.d + ROWS - 1) / ROWS);
        set_cursor<ROWS>(a, c, i / blocks, i % blocks);
    } else {
        const int th = last_at_most<THREADS>(l.seqs, (int64_t)i);
        const int32_t run = (a.sequences + THREADS - 1) / THREADS;
        set_cursor<ROWS>(a, c, th * run, 0);
        c.k = (int32_t)(i - l.seqs[th]);
        while (c.k >= c.blocks) {
            const int32_t k = c.k - c.blocks;
            set_cursor<ROWS>(a, c, c.b + 1, k);
        }
    }
    c.tiles = block_tiles<ROWS>(a, c.s, c.k);
    c.cost = c.tiles + unit_cost<ROWS>();
    return c;
}
// one sequence of a few blocks: every thread counts them all, without the two rounds through LDS (both launches, with
// the rounds : without: one token of a stream of 1000 11.9 : 10.5 us, over 16384 15.9 : 14.6; up to 64 blocks instead
// of 8 are counted no faster)
template <int ROWS>
__device__ inline bool few_blocks(const AttendArgs& a)
{
    return !a.starts && a.sequences == 1 && (uint32_t)a.per * a.by_group.d <= 8 * ROWS;
}
// all tiles, and the runs' sums in l.  Starts that do not ascend may claim tokens many times over: more blocks than
// there is room for in the pieces' list, or than 32 bits hold.  Such a call has no work, in every workgroup.
template <int THREADS, int ROWS>
__device__ inline int64_t count_work(const AttendArgs& a, Schedule<THREADS>& l, int32_t* all_blocks)
{
    if (few_blocks<ROWS>(a)) {
        Cursor c;
        set_cursor<ROWS>(a, c, 0, 0);
        int64_t sum = 0;
        for (int32_t k = 0; k < c.blocks; ++k) sum += block_tiles<ROWS>(a, c.s, k) + unit_cost<ROWS>();
        *all_blocks = c.blocks;
        return sum * a.c.heads;
    }
    int32_t blocks = 0;
    if (!a.starts) {
        blocks = a.sequences * (int32_t)(((uint32_t)a.per * a.by_group.d + ROWS - 1) / ROWS);
    } else {
        const int32_t run = (a.sequences + THREADS - 1) / THREADS;
        const int32_t b0 = min((int32_t)threadIdx.x * run, a.sequences), b1 = min(b0 + run, a.sequences);
        int64_t n = 0, all;
        for (int32_t b = b0; b < b1; ++b) n += seq_blocks<ROWS>(a, get_seq(a, b));
        group_scan<THREADS>(n, l.seqs, &all);
        if (all > a.most_blocks) {
            *all_blocks = 0;
            return 0;
        }
        blocks = (int32_t)all;
    }
    *all_blocks = blocks;
    const int32_t run = (blocks + THREADS - 1) / THREADS;
    const int32_t i0 = min((int32_t)threadIdx.x * run, blocks), i1 = min(i0 + run, blocks);
    int64_t w = 0, total;
    if (i0 < i1) {
        Cursor c = find_block<THREADS, ROWS>(a, l, i0);
        for (int32_t i = i0; i < i1; ++i) {
            w += c.cost;
            // not behind the last: the sequences of a padded batch that have no query would be walked one by one there
            // (8 of 256 sequences with a token each: 59 us instead of 18)
            if (i + 1 < i1) next_block<ROWS>(a, c);
        }
    }
    group_scan<THREADS>(w * a.c.heads, l.work, &total);
    return total;
}
// the block that has position `pos` of them all; before: the positions before that block, index: the blocks before it
template <int THREADS, int ROWS>
__device__ inline Cursor find_work(const AttendArgs& a, const Schedule<THREADS>& l, int32_t all_blocks, int64_t pos,
                                   int64_t* before, int32_t* index)
{
    const bool few = few_blocks<ROWS>(a);
    const int th = few ? 0 : last_at_most<THREADS>(l.work, pos);
    const int32_t run = (all_blocks + THREADS - 1) / THREADS;
    Cursor c;
    if (few) {
        set_cursor<ROWS>(a, c, 0, 0);
        c.tiles = block_tiles<ROWS>(a, c.s, 0);
        c.cost = c.tiles + unit_cost<ROWS>();
    } else {
        c = find_block<THREADS, ROWS>(a, l, th * run);
    }
    int64_t at = few ? 0 : l.work[th];
    *index = th * run;
    while (pos >= at + (int64_t)c.cost * a.c.heads) {
        at += (int64_t)c.cost * a.c.heads;
        ++*index;
        next_block<ROWS>(a, c);
    }
    *before = at;
    return c;
}

// the largest, or the sum, of x over the four lanes of a query (16 apart)
__device__ inline float query_max(float x)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float query_sum(float x)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A query's running maximum after scores of at most `top`.  Each query decides by itself: raised along with another of
// its wavefront, it would be rounded otherwise, and a token that only the other sees would show in its result.
__device__ inline float raised(float m, float top) { return top > m + kRaise ? top : m; }

// the largest of eight, a NaN left out: the median of two numbers and infinity is their maximum, and takes its
// operands as they are (the library's maximum first quiets what could be a signalling NaN: four instructions more)
__device__ inline float max8(const float* x)
{
    const float inf = __builtin_inff();
    const float a = __builtin_amdgcn_fmed3f(x[0], x[1], inf), b = __builtin_amdgcn_fmed3f(x[2], x[3], inf);
    const float c = __builtin_amdgcn_fmed3f(x[4], x[5], inf), d = __builtin_amdgcn_fmed3f(x[6], x[7], inf);
    return __builtin_amdgcn_fmed3f(__builtin_amdgcn_fmed3f(a, b, inf), __builtin_amdgcn_fmed3f(c, d, inf), inf);
}

// What a query's output is multiplied by: its last token is `limit` (below 0: it sees none, and gets 0).  A sum of 0
// else means that all its scores are minus infinity, which have no softmax.
__device__ inline float inverse_sum(float sum, int64_t limit)
{
    return sum != 0.0f ? 1.0f / sum : limit < 0 ? 0.0f : __builtin_nanf("");
}

// x as a sum of bf16 numbers, truncated one after the other (three hold all of fp32's 24 bits; the last of two
// is rounded to nearest): eight values into an operand for each part
template <int PARTS>
__device__ inline void split8(const float* x, bf16x8* part)
{
    u32x4 w[PARTS];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            if (p == PARTS - 1) {
                if constexpr (PARTS == 3) {
                    w[p][i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
                } else {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    w[p][i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
                }
            } else {
                w[p][i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
                a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
                b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) part[p] = __builtin_bit_cast(bf16x8, w[p]);
}

// The scale that byte k of x stands for.  The conversions of 8- and 4-bit floats read its exponent bits alone (255:
// NaN), so one shift brings it there; an integer is multiplied and needs the rest clear (255: infinity, times code 0).
template <int FMT, int K>
__device__ inline float scale_of(uint32_t x)
{
    if constexpr (FMT == SNACK_INT8) return __uint_as_float((x >> (8 * K) & 0xFFu) << 23);
    if constexpr (K == 0) return __uint_as_float(x << 23);
    if constexpr (K == 1) return __uint_as_float(x << 15);
    if constexpr (K == 2) return __uint_as_float(x << 7);
    return __uint_as_float(x >> 1);
}
__device__ inline uint32_t pack_bf16(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
template <int FMT, int HALF>   // two codes of a word's 16-bit half
__device__ inline uint32_t decode_half(uint32_t w, float scale)
{
    if constexpr (FMT == SNACK_E4M3)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HALF != 0));
    return pack_bf16((float)(int8_t)(w >> (16 * HALF) & 0xFFu) * scale, (float)(int8_t)(w >> (16 * HALF + 8) & 0xFFu) * scale);
}
template <int BYTE>   // two codes of a byte
__device__ inline uint32_t decode_byte(uint32_t w, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, BYTE));
}

// What a lane holds of a tile, as it lies in memory.
template <int FMT, int NB>
struct RawTile {
    static constexpr int KW = four_bits(FMT) ? 1 : 2;   // words of a K operand
    static constexpr int VW = four_bits(FMT) ? 2 : 4;   // words of a V block
    static constexpr int KE = NB <= 4 ? 1 : 2;          // words of a token's K exponents
    uint32_t k[2][NB * KW];
    uint32_t ke[2][KE];
    uint32_t v[NB * VW];
    uint32_t ve[NB * 2];
};
template <int N>
__device__ inline void load_words(uint32_t* w, const uint8_t* p)
{
    typedef uint32_t vec __attribute__((ext_vector_type(N), aligned(4)));
    const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = v[i];
}
template <>
__device__ inline void load_words<1>(uint32_t* w, const uint8_t* p)
{
    w[0] = *reinterpret_cast<const uint32_t*>(p);
}
// words W a block of a chunked array: 16 bytes a lane, kilobyte after kilobyte, the last chunk shorter
template <int NB, int W>
__device__ inline void load_chunks(uint32_t* w, const uint8_t* p, int lane)
{
    constexpr int per = 4 / W, full = NB / per, rest = NB % per;
#pragma unroll
    for (int c = 0; c < full; ++c) load_words<4>(w + 4 * c, p + 1024 * c + 16 * lane);
    if constexpr (rest > 0) load_words<rest * W>(w + 4 * full, p + 1024 * full + 4 * rest * W * lane);
}
template <int FMT, int NB>
__device__ inline void load_tile(RawTile<FMT, NB>& r, const uint8_t* tile, int lane)
{
    using R = RawTile<FMT, NB>;
    constexpr int half = kTile / 2 * NB * 4 * R::KW * 4 ;
    load_chunks<NB, R::KW>(r.k[0], tile, lane);
    load_chunks<NB, R::KW>(r.k[1], tile + half, lane);
    load_chunks<NB, R::VW>(r.v, tile + code_bytes(FMT, NB), lane);
    const uint8_t* e = tile + 2 * code_bytes(FMT, NB);
    constexpr int eb = k_exp_bytes(NB);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint8_t* p = e + (16 * s + (lane & 15)) * eb;
        if constexpr (eb == 1) r.ke[s][0] = *p;
        else if constexpr (eb == 2) r.ke[s][0] = *reinterpret_cast<const uint16_t*>(p);
        else load_words<R::KE>(r.ke[s], p);
    }
    const uint8_t* ev = e + kTile * eb + (lane >> 4) * NB * 8;
    constexpr int n4 = NB / 2;
#pragma unroll
    for (int i = 0; i < n4; ++i) load_words<4>(r.ve + 4 * i, ev + 16 * i);
    if constexpr (NB % 2) load_words<2>(r.ve + 4 * n4, ev + 16 * n4);
}

// the K operand of a block: its words, and the exponent in byte BYTE of e
template <int FMT, int BYTE>
__device__ inline bf16x8 key_operand(const uint32_t* k, uint32_t e)
{
    const float s = scale_of<FMT, BYTE>(e);
    u32x4 o;
    if constexpr (four_bits(FMT)) {
        o = u32x4{decode_byte<0>(k[0], s), decode_byte<1>(k[0], s), decode_byte<2>(k[0], s), decode_byte<3>(k[0], s)};
    } else {
        o = u32x4{decode_half<FMT, 0>(k[0], s), decode_half<FMT, 1>(k[0], s), decode_half<FMT, 0>(k[1], s),
                  decode_half<FMT, 1>(k[1], s)};
    }
    return __builtin_bit_cast(bf16x8, o);
}
// the V operands of a block: features 0..15 of it, and 16..31
template <int FMT>
__device__ inline void value_operands(const uint32_t* v, const uint32_t* ve, bf16x8& lo, bf16x8& hi)
{
    const uint32_t e0 = ve[0], e1 = ve[1];
    const float s[8] = {scale_of<FMT, 0>(e0), scale_of<FMT, 1>(e0), scale_of<FMT, 2>(e0), scale_of<FMT, 3>(e0),
                        scale_of<FMT, 0>(e1), scale_of<FMT, 1>(e1), scale_of<FMT, 2>(e1), scale_of<FMT, 3>(e1)};
    u32x4 a, b;
    if constexpr (FMT == SNACK_INT8) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t w = v[r];
            a[r] = pack_bf16((float)(int8_t)(w & 0xFFu) * s[2 * r], (float)(int8_t)(w >> 16 & 0xFFu) * s[2 * r + 1]);
            b[r] = pack_bf16((float)(int8_t)(w >> 8 & 0xFFu) * s[2 * r], (float)(int8_t)(w >> 24) * s[2 * r + 1]);
        }
    } else {
        uint32_t w[8];   // both features of one token each
        if constexpr (four_bits(FMT)) {
            const uint32_t x = v[0], y = v[1];
            w[0] = decode_byte<0>(x, s[0]); w[1] = decode_byte<1>(x, s[1]);
            w[2] = decode_byte<2>(x, s[2]); w[3] = decode_byte<3>(x, s[3]);
            w[4] = decode_byte<0>(y, s[4]); w[5] = decode_byte<1>(y, s[5]);
            w[6] = decode_byte<2>(y, s[6]); w[7] = decode_byte<3>(y, s[7]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[2 * r] = decode_half<FMT, 0>(v[r], s[2 * r]);
                w[2 * r + 1] = decode_half<FMT, 1>(v[r], s[2 * r + 1]);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            a[r] = __builtin_amdgcn_perm(w[2 * r + 1], w[2 * r], 0x05040100u);
            b[r] = __builtin_amdgcn_perm(w[2 * r + 1], w[2 * r], 0x07060302u);
        }
    }
    lo = __builtin_bit_cast(bf16x8, a);
    hi = __builtin_bit_cast(bf16x8, b);
}

// f(0), f(1), ..., f(N - 1) with the index a constant
template <int N, typename F>
__device__ inline void unroll(F f)
{
    if constexpr (N > 0) {
        unroll<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// the first n of 8 tokens' bytes of a word pair kept, n within 0..8
__device__ inline uint64_t first_bytes(int n) { return n >= 8 ? ~0ull : n <= 0 ? 0ull : (1ull << (8 * n)) - 1; }

// how many of the lane's eight tokens base + 8 g + 0..7 come up to `limit`
__device__ inline int tokens_seen(int64_t limit, int64_t base, int g)
{
    const int64_t n = limit - base - 8 * g + 1;
    return n > 8 ? 8 : n < 0 ? 0 : (int)n;
}

// A V block's codes and exponents of the tokens whose byte is not in m become 0.
template <int FMT>
__device__ inline void clear_block(uint32_t* v, uint32_t* ve, uint64_t m)
{
    const uint32_t m0 = (uint32_t)m, m1 = (uint32_t)(m >> 32);
    ve[0] &= m0;
    ve[1] &= m1;
    if constexpr (four_bits(FMT)) {
        v[0] &= m0;
        v[1] &= m1;
    } else {
        // two bytes a token
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = (i < 2 ? m0 : m1) >> (16 * (i & 1));
            v[i] &= (x & 0xFFu ? 0xFFFFu : 0u) | (x & 0xFF00u ? 0xFFFF0000u : 0u);
        }
    }
}
// The tokens of the tile (a bit each, the same in every lane) whose exponent byte in this V block is 255, which
// becomes 0 (their codes are 0).
__device__ inline uint32_t take_nans(uint32_t* ve)
{
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = ~ve[i];
        any |= (x - 0x01010101u) & ~x & 0x80808080u;
    }
    if (__ballot(any != 0) == 0) return 0;
    uint64_t e = (uint64_t)ve[1] << 32 | ve[0];
    uint32_t tokens = 0;
    for (int j = 0; j < 8; ++j) {
        const bool is = (e >> (8 * j) & 0xFFu) == 255u;
        if (is) e &= ~(0xFFull << (8 * j));
        const uint64_t m = __ballot(is);
        for (int g = 0; g < 4; ++g) tokens |= (uint32_t)(m >> (16 * g) & 1) << (8 * g + j);
    }
    ve[0] = (uint32_t)e;
    ve[1] = (uint32_t)(e >> 32);
    return tokens;
}

// one query's row of the output: token and query head of query `row` of cache head h
struct Row {
    int32_t i, head;   // index among the sequence's tokens; the query head
};
__device__ inline Row get_row(const AttendArgs& a, int32_t h, uint32_t row)
{
    const uint32_t i = fast_quot(a.by_group, row);
    return Row{(int32_t)i, (int32_t)(h * a.by_group.d + (row - i * a.by_group.d))};
}

// features f0 + 32 j + 0..7 of a head of d, j < NB, without a branch round each load: where d is a multiple of 8, what
// is past it is read from the head's start and left out
template <int NB, typename Q>
__device__ inline void load_query(f32x8* x, const Q* __restrict__ p, int f0, int d)
{
    if (d % 8 == 0) {
#pragma unroll
        for (int j = 0; j < NB; ++j) x[j] = load8(p + (f0 + 32 * j < d ? f0 + 32 * j : 0), 8);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (f0 + 32 * j >= d) x[j] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    } else {
#pragma unroll
        for (int j = 0; j < NB; ++j) x[j] = load8(p + f0 + 32 * j, d - f0 - 32 * j);
    }
}
// and their parts as operands
template <int PARTS, int NB>
__device__ inline void split_query(bf16x8 (*q)[NB], const f32x8* x)
{
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[j][i];
        bf16x8 part[PARTS];
        split8<PARTS>(y, part);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) q[k][j] = part[k];
    }
}

// x / d rounded down, for 0 <= x < 2^52: the quotient in floating point is off by one at most
__device__ inline int64_t divide(int64_t x, int64_t d)
{
    int64_t q = (int64_t)((double)x / (double)d);
    q -= q * d > x ? 1 : 0;
    return q + (x - q * d >= d ? 1 : 0);
}

template <int QT>
struct QType { using T = float; };
template <>
struct QType<SNACK_BF16> { using T = uint16_t; };

// four features d.. of an output row
template <int QT>
__device__ inline void store_out(void* out, int64_t at, int d, int dims, f32x4 v)
{
    if constexpr (QT == SNACK_F32) {
        float* p = (float*)out + at + d;
        if (d + 4 <= dims) *reinterpret_cast<f32x4u*>(p) = v;
        else
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (d + i < dims) p[i] = v[i];
    } else {
        uint16_t* p = (uint16_t*)out + at + d;
        if (d + 4 <= dims) *reinterpret_cast<u16x4u*>(p) = u16x4u{bf16_bits(v.x), bf16_bits(v.y), bf16_bits(v.z), bf16_bits(v.w)};
        else
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (d + i < dims) p[i] = bf16_bits(v[i]);
    }
}

// The pieces of a unit (blockIdx.x: the unit, or the workgroup that started it), joined: 16 queries (blockIdx.y).  WIDE
// (few units of many pieces each): 16 features (blockIdx.z), the wavefronts sharing the pieces out; else every wavefront
// some of the features, over all pieces.  A chain of three loads bounds it: the unit, its pieces' maxima, sums and
// outputs all at once, the result (4 to 5 us with its launch; 40 MB of pieces in 9.5 us).
template <int QT, int ROWS, bool WIDE>
__global__ void __launch_bounds__(kAttendThreads) attend_join_kernel(AttendArgs a)
{
    __shared__ float red[kAttendThreads / kQueries][kQueries];
    __shared__ f32x4 so[kAttendWaves][kWave];
    if (a.by_unit && (int)blockIdx.x >= a.meta[a.meta_last].x) return;
    const int4 u = a.meta[2 * blockIdx.x], u1 = a.meta[2 * blockIdx.x + 1];
    const uint32_t rows = (uint32_t)u1.x, row0 = (uint32_t)u.y * ROWS + 16 * blockIdx.y;
    if (u.w == 0 || row0 >= rows) return;
    const int lane = (int)threadIdx.x & (kWave - 1), wave = (int)threadIdx.x / kWave;
    const int col = lane & 15, g = lane >> 4;
    const int size = part_floats(a.c.nb), pieces = u.w, tail = 2 * a.c.nb * 256 + 2 * col;
    const int i0 = WIDE ? (int)blockIdx.z : wave;     // the first 16 features
    const bool seen = row0 + col < rows, live = seen && i0 < 2 * a.c.nb;
    // piece k's results of these queries
    auto piece = [&](int k) {
        return a.part + ((int64_t)(2 * (u1.y + k) + (k == 0 ? 1 : 0)) * (ROWS / 16) + blockIdx.y) * size;
    };
    auto output = [&](int k, int i) { return *reinterpret_cast<const f32x4*>(piece(k) + (i * kWave + lane) * 4); };
    // The loads of the first pieces, all at once: each of a chain of loads would take a microsecond.
    constexpr int kStep = kAttendThreads / kQueries, kMl = 4;     // threads of a query, their pieces
    constexpr int kX = WIDE ? 16 : 4;
    const int first = (int)threadIdx.x / kQueries, k0 = WIDE ? wave : 0, ks = WIDE ? kAttendWaves : 1;
    float2 ml[kMl];
    f32x4 x[kX];
    float xm[kX];        // their maxima: a weight is made where it is used (a list of them in LDS keeps workgroups out)
#pragma unroll
    for (int r = 0; r < kMl; ++r) {
        const int k = first + kStep * r;
        ml[r] = seen && k < pieces ? *reinterpret_cast<const float2*>(piece(k) + tail) : make_float2(-__builtin_inff(), 0.0f);
    }
#pragma unroll
    for (int r = 0; r < kX; ++r) {
        const int k = k0 + ks * r;
        x[r] = live && k < pieces ? output(k, i0) : f32x4{0, 0, 0, 0};
        xm[r] = live && k < pieces ? piece(k)[tail] : -__builtin_inff();
    }
    float m = -__builtin_inff();
#pragma unroll
    for (int r = 0; r < kMl; ++r) m = fmaxf(m, ml[r].x);
    if (seen)
        for (int k = first + kStep * kMl; k < pieces; k += kStep) m = fmaxf(m, piece(k)[tail]);
    red[first][col] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStep; ++i) m = fmaxf(m, red[i][col]);
    __syncthreads();
    const float off = m == -__builtin_inff() ? 0.0f : m;
    float sum = 0.0f;
    auto weight = [&](float top) { return __builtin_amdgcn_exp2f(top - off); };
#pragma unroll
    for (int r = 0; r < kMl; ++r) sum = fmaf(weight(ml[r].x), ml[r].y, sum);
    if (seen)
        for (int k = first + kStep * kMl; k < pieces; k += kStep) {
            const float2 p = *reinterpret_cast<const float2*>(piece(k) + tail);
            sum = fmaf(weight(p.x), p.y, sum);
        }
    red[first][col] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kStep; ++i) sum += red[i][col];
    const Row mine = get_row(a, u.z, min(row0 + col, rows - 1));
    const float inv = inverse_sum(sum, a.causal ? u1.z + mine.i : u1.z);
    const int64_t at = ((int64_t)(u.x + mine.i) * a.hq + mine.head) * a.c.d;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < kX; ++r) v += x[r] * weight(xm[r]);
    if (live)
        for (int k = k0 + ks * kX; k < pieces; k += ks) v += output(k, i0) * weight(piece(k)[tail]);
    if constexpr (WIDE) {
        so[wave][lane] = v;
        __syncthreads();
        if (wave != 0 || !live) return;
#pragma unroll
        for (int w = 1; w < kAttendWaves; ++w) v += so[w][lane];
        store_out<QT>(a.out, at, 16 * i0 + 4 * g, a.c.d, v * inv);
    } else {
        if (!live) return;
        for (int i = i0;;) {
            store_out<QT>(a.out, at, 16 * i + 4 * g, a.c.d, v * inv);
            i += kAttendWaves;
            if (i >= 2 * a.c.nb) break;
            v = f32x4{0, 0, 0, 0};
#pragma unroll 4
            for (int k = 0; k < pieces; ++k) v += output(k, i) * weight(piece(k)[tail]);
        }
    }
}

// which kernel: by the queries of a block
enum AttendKind : int { kFew = 0, kMany64, kMany256 };
constexpr int attend_rows(int kind) { return kQueries << (2 * kind); }

// one file a format: attend_int8.hip, attend_e4m3.hip, attend_e2m1.hip
template <int FMT>
snack_status launch_attend(const AttendArgs& a, int q_fmt, int kind, unsigned groups, hipStream_t s);
extern template snack_status launch_attend<SNACK_INT8>(const AttendArgs&, int, int, unsigned, hipStream_t);
extern template snack_status launch_attend<SNACK_E4M3>(const AttendArgs&, int, int, unsigned, hipStream_t);
extern template snack_status launch_attend<SNACK_E2M1>(const AttendArgs&, int, int, unsigned, hipStream_t);

}  // namespace snack
