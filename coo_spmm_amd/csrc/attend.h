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
// layout); every cached value is exactly a bf16 number.  An fp32 query is split into
// three bf16 numbers whose sum it is, and so is every probability: three exact
// products added in fp32, for which there is room, since the cache's bytes bound
// this kernel.  With bf16 queries the probabilities keep 16 bits (two numbers).
//
// Work is cut without regard to the sequences' ends: all (sequence, head, queries)
// units one after the other are a row of tiles, of which every workgroup takes an
// equal run, its four wavefronts taking tiles in turn.  So one long sequence among
// short ones fills the card like any other batch.  A unit that one workgroup has
// whole is written by it; the pieces of the others are joined by a second launch in
// a fixed order.
#pragma once

#include "cache.h"
#include "rope.h"

namespace snack {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttendWaves = 4;
constexpr int kAttendThreads = kAttendWaves * kWave;
constexpr int kQueries = 16;          // queries of a unit
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
    int32_t hq;
    FastDiv by_group;                 // query heads of a cache head
    float scale_log2;                 // scale * log2(e)
    int32_t causal;
    float* part;                      // two partial results a workgroup: of the block it goes on with, of the one it starts
    int4* meta;                       // of the block a workgroup starts and does not end: sequence, block, head, pieces
};

// floats of a partial result of 16 queries: the output's, then maximum and sum of every query
__host__ __device__ constexpr int part_floats(int nb) { return 2 * nb * 256 + 2 * kQueries; }

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
        s.first = min(max(a.starts[b], 0), a.tokens);
        last = min(max(a.starts[b + 1], s.first), a.tokens);
    } else {
        s.first = b * a.per;
        last = s.first + a.per;
    }
    s.nq = last - s.first;
    s.len = max(a.lens[b], 0);
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

// The work: for every sequence, every block of queries, every cache head, the block's tiles, all one after the other.
// Where a position of this row lies:
struct Cursor {
    int32_t b, k;             // sequence, block
    int32_t blocks, tiles;    // of the sequence, of the block (of every head of it)
    Seq s;
};
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
    int32_t seqs[THREADS + THREADS / kWave];   // blocks before a thread's run of sequences
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
        const int th = last_at_most<THREADS>(l.seqs, i);
        const int32_t run = (a.sequences + THREADS - 1) / THREADS;
        set_cursor<ROWS>(a, c, th * run, 0);
        c.k = i - l.seqs[th];
        while (c.k >= c.blocks) {
            const int32_t k = c.k - c.blocks;
            set_cursor<ROWS>(a, c, c.b + 1, k);
        }
    }
    c.tiles = block_tiles<ROWS>(a, c.s, c.k);
    return c;
}
// all tiles, and the runs' sums in l
template <int THREADS, int ROWS>
__device__ inline int64_t count_work(const AttendArgs& a, Schedule<THREADS>& l, int32_t* all_blocks)
{
    int32_t blocks = 0;
    if (!a.starts) {
        blocks = a.sequences * (int32_t)(((uint32_t)a.per * a.by_group.d + ROWS - 1) / ROWS);
    } else {
        const int32_t run = (a.sequences + THREADS - 1) / THREADS;
        const int32_t b0 = min((int32_t)threadIdx.x * run, a.sequences), b1 = min(b0 + run, a.sequences);
        int32_t n = 0;
        for (int32_t b = b0; b < b1; ++b) n += seq_blocks<ROWS>(a, get_seq(a, b));
        group_scan<THREADS>(n, l.seqs, &blocks);
    }
    *all_blocks = blocks;
    const int32_t run = (blocks + THREADS - 1) / THREADS;
    const int32_t i0 = min((int32_t)threadIdx.x * run, blocks), i1 = min(i0 + run, blocks);
    int64_t w = 0, total;
    if (i0 < i1) {
        Cursor c = find_block<THREADS, ROWS>(a, l, i0);
        for (int32_t i = i0; i < i1; ++i) {
            w += c.tiles;
            next_block<ROWS>(a, c);
        }
    }
    group_scan<THREADS>(w * a.c.heads, l.work, &total);
    return total;
}
// the block that has tile `pos` of them all; before: the tiles before that block
template <int THREADS, int ROWS>
__device__ inline Cursor find_work(const AttendArgs& a, const Schedule<THREADS>& l, int32_t all_blocks, int64_t pos,
                                   int64_t* before)
{
    const int th = last_at_most<THREADS>(l.work, pos);
    const int32_t run = (all_blocks + THREADS - 1) / THREADS;
    Cursor c = find_block<THREADS, ROWS>(a, l, th * run);
    int64_t at = l.work[th];
    while (pos >= at + (int64_t)c.tiles * a.c.heads) {
        at += (int64_t)c.tiles * a.c.heads;
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

// the K operand of block J of a half
template <int FMT, int NB, int J>
__device__ inline bf16x8 key_operand(const uint32_t* k, const uint32_t* ke)
{
    const float s = scale_of<FMT, J % 4>(ke[J / 4]);
    u32x4 o;
    if constexpr (four_bits(FMT)) {
        const uint32_t w = k[J];
        o = u32x4{decode_byte<0>(w, s), decode_byte<1>(w, s), decode_byte<2>(w, s), decode_byte<3>(w, s)};
    } else {
        const uint32_t a = k[2 * J], b = k[2 * J + 1];
        o = u32x4{decode_half<FMT, 0>(a, s), decode_half<FMT, 1>(a, s), decode_half<FMT, 0>(b, s),
                  decode_half<FMT, 1>(b, s)};
    }
    return __builtin_bit_cast(bf16x8, o);
}
// the V operands of block B: features 0..15 of it, and 16..31
template <int FMT, int NB, int B>
__device__ inline void value_operands(const uint32_t* v, const uint32_t* ve, bf16x8& lo, bf16x8& hi)
{
    const uint32_t e0 = ve[2 * B], e1 = ve[2 * B + 1];
    const float s[8] = {scale_of<FMT, 0>(e0), scale_of<FMT, 1>(e0), scale_of<FMT, 2>(e0), scale_of<FMT, 3>(e0),
                        scale_of<FMT, 0>(e1), scale_of<FMT, 1>(e1), scale_of<FMT, 2>(e1), scale_of<FMT, 3>(e1)};
    u32x4 a, b;
    if constexpr (FMT == SNACK_INT8) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t w = v[4 * B + r];
            a[r] = pack_bf16((float)(int8_t)(w & 0xFFu) * s[2 * r], (float)(int8_t)(w >> 16 & 0xFFu) * s[2 * r + 1]);
            b[r] = pack_bf16((float)(int8_t)(w >> 8 & 0xFFu) * s[2 * r], (float)(int8_t)(w >> 24) * s[2 * r + 1]);
        }
    } else {
        uint32_t w[8];   // both features of one token each
        if constexpr (four_bits(FMT)) {
            const uint32_t x = v[2 * B], y = v[2 * B + 1];
            w[0] = decode_byte<0>(x, s[0]); w[1] = decode_byte<1>(x, s[1]);
            w[2] = decode_byte<2>(x, s[2]); w[3] = decode_byte<3>(x, s[3]);
            w[4] = decode_byte<0>(y, s[4]); w[5] = decode_byte<1>(y, s[5]);
            w[6] = decode_byte<2>(y, s[6]); w[7] = decode_byte<3>(y, s[7]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[2 * r] = decode_half<FMT, 0>(v[4 * B + r], s[2 * r]);
                w[2 * r + 1] = decode_half<FMT, 1>(v[4 * B + r], s[2 * r + 1]);
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

// The pieces of the unit that workgroup blockIdx.x of the first launch started, joined; 16 features (blockIdx.y) of 16
// queries (blockIdx.z).
template <int QT, int ROWS>
__global__ void __launch_bounds__(kAttendThreads) attend_join_kernel(AttendArgs a)
{
    __shared__ f32x4 so[kAttendWaves][kWave];
    __shared__ float2 sml[kAttendWaves][kQueries];
    const int4 u = a.meta[blockIdx.x];
    if (u.w == 0) return;
    const int lane = (int)threadIdx.x & (kWave - 1), wave = (int)threadIdx.x / kWave;
    const int col = lane & 15, g = lane >> 4, i = (int)blockIdx.y;
    const int size = part_floats(a.c.nb);
    const Seq s = get_seq(a, u.x);
    const int32_t h = u.z;
    const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row = (uint32_t)u.y * ROWS + 16 * blockIdx.z + col;
    const bool live = row < rows;
    float m = -__builtin_inff(), sum = 0.0f;
    f32x4 v = {0, 0, 0, 0};
    for (int k = wave; k < u.w; k += kAttendWaves) {
        const float* part = a.part + ((int64_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * (ROWS / 16) + blockIdx.z) * size;
        float2 ml = make_float2(-__builtin_inff(), 0.0f);
        f32x4 x = {0, 0, 0, 0};
        if (live) {
            ml = *reinterpret_cast<const float2*>(part + 2 * a.c.nb * 256 + 2 * col);
            x = *reinterpret_cast<const f32x4*>(part + (i * kWave + lane) * 4);
        }
        const float n = fmaxf(m, ml.x), ns = n == -__builtin_inff() ? 0.0f : n;
        const float f0 = __builtin_amdgcn_exp2f(m - ns), f1 = __builtin_amdgcn_exp2f(ml.x - ns);
        v = v * f0 + x * f1;
        sum = sum * f0 + ml.y * f1;
        m = n;
    }
    so[wave][lane] = v;
    if (g == 0) sml[wave][col] = make_float2(m, sum);
    __syncthreads();
    if (wave != 0 || !live) return;
    m = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kAttendWaves; ++w) m = fmaxf(m, sml[w][col].x);
    const float ms = m == -__builtin_inff() ? 0.0f : m;
    sum = 0.0f;
    v = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kAttendWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(sml[w][col].x - ms);
        sum = fmaf(f, sml[w][col].y, sum);
        v += so[w][lane] * f;
    }
    const Row mine = get_row(a, h, row);
    const int64_t at = ((int64_t)(s.first + mine.i) * a.hq + mine.head) * a.c.d;
    store_out<QT>(a.out, at, 16 * i + 4 * g, a.c.d, sum == 0.0f ? f32x4{0, 0, 0, 0} : v * (1.0f / sum));
}

enum AttendKind : int { kFew = 0, kMany64, kMany128 };
constexpr int attend_rows(int kind) { return kind == kFew ? kQueries : kind == kMany64 ? 64 : 128; }

// one file a format: attend_int8.hip, attend_e4m3.hip, attend_e2m1.hip
template <int FMT>
snack_status launch_attend(const AttendArgs& a, int q_fmt, int kind, unsigned groups, hipStream_t s);
extern template snack_status launch_attend<SNACK_INT8>(const AttendArgs&, int, int, unsigned, hipStream_t);
extern template snack_status launch_attend<SNACK_E4M3>(const AttendArgs&, int, int, unsigned, hipStream_t);
extern template snack_status launch_attend<SNACK_E2M1>(const AttendArgs&, int, int, unsigned, hipStream_t);

}  // namespace snack
