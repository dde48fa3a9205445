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
    float* part;                      // two partial results a workgroup: of the unit it goes on with, of the one it starts
    int4* meta;                       // of the unit a workgroup starts and does not end: sequence, unit in it, pieces
};

// floats of a partial result: the output's, then maximum and sum of every query
__host__ __device__ constexpr int part_floats(int nb) { return 2 * nb * 256 + 2 * kQueries; }

// a sequence of the call
struct Seq {
    int32_t first, nq, len;
    int32_t blocks;   // of kQueries queries of a cache head
    int32_t tiles;    // at least 1 (a query that sees nothing is still answered)
};
__device__ inline Seq get_seq(const AttendArgs& a, int32_t b, int rows)
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
    s.blocks = (int32_t)(((int64_t)s.nq * a.by_group.d + rows - 1) / rows);
    // tokens past the page table are one more tile, which stands for all of them
    const int64_t room = (int64_t)a.width * a.c.page_tiles + 1;
    const int64_t t = ((int64_t)s.len + kTile - 1) / kTile;
    s.tiles = (int32_t)(t < 1 ? 1 : t < room ? t : room);
    return s;
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

// The codes and exponents of the tokens past the first n of the lane's eight become 0.
template <int FMT, int NB>
__device__ inline void clear_values(RawTile<FMT, NB>& r, int n)
{
    const uint64_t m = first_bytes(n);
    const uint32_t m0 = (uint32_t)m, m1 = (uint32_t)(m >> 32);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        r.ve[2 * b] &= m0;
        r.ve[2 * b + 1] &= m1;
        if constexpr (four_bits(FMT)) {
            r.v[2 * b] &= m0;
            r.v[2 * b + 1] &= m1;
        } else {
            // two bytes a token
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = (i < 2 ? m0 : m1) >> (16 * (i & 1));
                r.v[4 * b + i] &= (x & 0xFFu ? 0xFFFFu : 0u) | (x & 0xFF00u ? 0xFFFF0000u : 0u);
            }
        }
    }
}

// Where position `pos` of the row of tiles lies: the sequence and the tiles of it before. The workgroup's threads
// take a run of sequences each; total: all tiles.
struct Spot {
    int32_t b;
    int64_t before;
};
template <int THREADS>
__device__ inline int64_t total_work(const AttendArgs& a, int rows, int64_t* sums)
{
    const int32_t run = (a.sequences + THREADS - 1) / THREADS;
    const int32_t b0 = min((int32_t)threadIdx.x * run, a.sequences), b1 = min(b0 + run, a.sequences);
    int64_t w = 0;
    for (int32_t b = b0; b < b1; ++b) {
        const Seq s = get_seq(a, b, rows);
        w += (int64_t)a.c.heads * s.blocks * s.tiles;
    }
    // inclusive sums over the threads
    int64_t x = w;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int64_t y = __shfl_up(x, d, kWave);
        if (((int)threadIdx.x & (kWave - 1)) >= d) x += y;
    }
    const int wave = (int)threadIdx.x / kWave;
    if (((int)threadIdx.x & (kWave - 1)) == kWave - 1) sums[THREADS + wave] = x;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) {
        if (i == wave) x += total;
        total += sums[THREADS + i];
    }
    sums[threadIdx.x] = x - w;   // before this thread's run
    __syncthreads();
    return total;
}
template <int THREADS>
__device__ inline Spot find_spot(const AttendArgs& a, int rows, const int64_t* sums, int64_t pos)
{
    // the last thread whose run starts at or before pos, then the sequences of its run (the runs past the last
    // sequence are empty and start at the total, which is past pos)
    int lo = 0, hi = THREADS - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (sums[m] <= pos) lo = m;
        else hi = m - 1;
    }
    const int32_t run = (a.sequences + THREADS - 1) / THREADS;
    Spot at{lo * run, sums[lo]};
    for (;;) {
        const Seq s = get_seq(a, at.b, rows);
        const int64_t w = (int64_t)a.c.heads * s.blocks * s.tiles;
        if (pos < at.before + w || at.b + 1 >= a.sequences) return at;
        at.before += w;
        ++at.b;
    }
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

// Values of a tile in which some query does not see some token: what has the exponent byte 255 is NaN, and a query
// that gives it the weight 0 because it does not see it must not get 0 NaN.  Their exponents become 0 (codes are 0),
// and the queries that do see them get their NaN here.
template <int FMT, int NB>
__device__ inline void nan_values(RawTile<FMT, NB>& r, f32x4* o, int64_t base, int64_t limit)
{
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
        const uint32_t x = ~r.ve[i];
        any |= (x - 0x01010101u) & ~x & 0x80808080u;
    }
    if (__ballot(any != 0) == 0) return;
    unroll<NB>([&](auto bc) {
        constexpr int b = decltype(bc)::value;
        const uint64_t e = (uint64_t)r.ve[2 * b + 1] << 32 | r.ve[2 * b];
        uint64_t kept = e;
        for (int j = 0; j < 8; ++j) {
            const bool is = (e >> (8 * j) & 0xFFu) == 255u;
            if (is) kept &= ~(0xFFull << (8 * j));
            const uint64_t m = __ballot(is);
            for (int g = 0; g < 4; ++g)
                if ((m >> (16 * g) & 1) && base + 8 * g + j <= limit) {
                    const float nan = __builtin_nanf("");
                    o[2 * b] = o[2 * b + 1] = f32x4{nan, nan, nan, nan};
                }
        }
        r.ve[2 * b] = (uint32_t)kept;
        r.ve[2 * b + 1] = (uint32_t)(kept >> 32);
    });
}

template <int FMT, int NB, int QT>
__global__ void __launch_bounds__(kAttendThreads, NB <= 4 ? 2 : 1) attend_kernel(AttendArgs a)
{
    constexpr int QP = QT == SNACK_F32 ? 3 : 1, PP = QT == SNACK_F32 ? 3 : 2;
    using Q = typename QType<QT>::T;
    __shared__ int64_t sums[kAttendThreads + kAttendWaves];
    __shared__ f32x4 so[kAttendWaves][2 * NB][kWave];
    __shared__ float2 sml[kAttendWaves][kQueries];
    const int lane = (int)threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int col = lane & 15, g = lane >> 4;

    const int64_t total = total_work<kAttendThreads>(a, kQueries, sums);
    int64_t run = (total + gridDim.x - 1) / gridDim.x;
    if (run < kMinRun) run = kMinRun;
    int64_t pos = run * blockIdx.x;
    const int64_t end = min(total, pos + run);
    if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (pos >= end) return;
    const Spot spot = find_spot<kAttendThreads>(a, kQueries, sums, pos);
    int32_t b = __builtin_amdgcn_readfirstlane(spot.b);
    Seq s = get_seq(a, b, kQueries);
    int64_t within = pos - spot.before;   // tiles of the sequence's units before pos
    int32_t unit = (int32_t)(within / s.tiles);
    int32_t t0 = (int32_t)(within - (int64_t)unit * s.tiles);

    while (pos < end) {
        // sequences without a query have no unit
        while (unit >= a.c.heads * s.blocks) {
            unit = 0;
            s = get_seq(a, ++b, kQueries);
        }
        const int32_t h = unit / s.blocks, block = unit - h * s.blocks;
        const int32_t t1 = (int32_t)min((int64_t)s.tiles, t0 + (end - pos));
        const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row0 = (uint32_t)block * kQueries;
        const uint32_t row = row0 + col;
        const bool live = row < rows;
        const Row mine = get_row(a, h, live ? row : rows - 1);
        // the last token a query sees, of this lane's and of the unit's first
        const int64_t past = a.causal ? (int64_t)s.len - s.nq : (int64_t)s.len - 1;
        const int64_t limit = a.causal ? past + mine.i : past;
        const int64_t least = a.causal ? past + fast_quot(a.by_group, row0) : past;

        bf16x8 q[QP][NB];
        {
            const Q* p = (const Q*)a.q + (int64_t)(s.first + mine.i) * a.q_row + (int64_t)mine.head * a.q_head + 8 * g;
            unroll<NB>([&](auto jc) {
                constexpr int j = decltype(jc)::value;
                const f32x8 x = load8(p + 32 * j, a.c.d - 8 * g - 32 * j);
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i];
                bf16x8 part[QP];
                split8<QP>(y, part);
#pragma unroll
                for (int k = 0; k < QP; ++k) q[k][j] = part[k];
            });
        }

        f32x4 o[2 * NB];
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) o[i] = f32x4{0, 0, 0, 0};
        float mc = -__builtin_inff(), l = 0.0f;   // running maximum times scale_log2; this lane's sum

        const int32_t* pages = a.table + (int64_t)b * a.width;
        auto page_of = [&](int32_t t) {
            const int32_t p = (int32_t)fast_quot(a.c.by_page, (uint32_t)t);
            return p < a.width ? pages[p] : -1;
        };
        auto tile_at = [&](int32_t t, int32_t page) {
            const uint32_t p = fast_quot(a.c.by_page, (uint32_t)t);
            const bool ok = page >= 0 && page < a.pages;
            return a.c.data + (int64_t)(ok ? page : 0) * a.c.page_bytes +
                   ((int64_t)h * a.c.page_tiles + (t - p * a.c.page_tiles)) * a.c.record;
        };
        RawTile<FMT, NB> cur, next;
        int32_t t = t0 + wave;
        int32_t page = 0, page1 = 0;
        if (t < t1) {
            page = page_of(t);
            page1 = page_of(min(t + kAttendWaves, t1 - 1));
            load_tile(cur, tile_at(t, page), lane);
        }
        for (; t < t1; t += kAttendWaves) {
            const int32_t tn = min(t + kAttendWaves, t1 - 1);
            load_tile(next, tile_at(tn, page1), lane);
            const int32_t page2 = page_of(min(t + 2 * kAttendWaves, t1 - 1));
            const int64_t base = (int64_t)t * kTile;
            const bool bad = page < 0 || page >= a.pages;
            f32x4 sc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
            unroll<NB>([&](auto jc) {
                constexpr int j = decltype(jc)::value;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const bf16x8 k = key_operand<FMT, NB, j>(cur.k[half], cur.ke[half]);
#pragma unroll
                    for (int i = QP - 1; i >= 0; --i)
                        sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[i][j], sc[half], 0, 0, 0);
                }
            });
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][i & 3];
            if (bad || base + kTile - 1 > least) {
                if (bad) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
                    clear_values(cur, 0);
                } else {
                    const int64_t left = (int64_t)s.len - base - 8 * g;
                    clear_values(cur, left > 8 ? 8 : left < 0 ? 0 : (int)left);
                    if (a.causal) nan_values(cur, o, base, live ? limit : -1);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (base + 8 * g + i > limit) x[i] = -__builtin_inff();
            }
            const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                                    fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * a.scale_log2;
            if (__ballot(top > mc + kRaise)) {
                const float m = fmaxf(mc, query_max(top));
                const float f = m == mc ? 1.0f : __builtin_amdgcn_exp2f(mc - m);
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) o[i] *= f;
                l *= f;
                mc = m;
            }
            const float off = mc == -__builtin_inff() ? 0.0f : -mc;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], a.scale_log2, off));
                l += x[i];
            }
            bf16x8 p[PP];
            split8<PP>(x, p);
            unroll<NB>([&](auto bc) {
                constexpr int blk = decltype(bc)::value;
                bf16x8 lo, hi;
                value_operands<FMT, NB, blk>(cur.v, cur.ve, lo, hi);
#pragma unroll
                for (int i = PP - 1; i >= 0; --i) {
                    o[2 * blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, p[i], o[2 * blk], 0, 0, 0);
                    o[2 * blk + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, p[i], o[2 * blk + 1], 0, 0, 0);
                }
            });
            cur = next;
            page = page1;
            page1 = page2;
        }
        // the wavefronts' results of the unit, joined
        l = query_sum(l);
        if (g == 0) sml[wave][col] = make_float2(mc, l);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) so[wave][i][lane] = o[i];
        __syncthreads();
        float m = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) m = fmaxf(m, sml[w][col].x);
        const float ms = m == -__builtin_inff() ? 0.0f : m;
        float f[kAttendWaves], sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) {
            f[w] = __builtin_amdgcn_exp2f(sml[w][col].x - ms);
            sum = fmaf(f[w], sml[w][col].y, sum);
        }
        const bool whole = t0 == 0 && t1 == s.tiles;
        float* part = a.part + (int64_t)(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * part_floats(NB);
        const int64_t at = ((int64_t)(s.first + mine.i) * a.hq + mine.head) * a.c.d;
        const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
        for (int i = wave; i < 2 * NB; i += kAttendWaves) {
            f32x4 v = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) v += so[w][i][lane] * f[w];
            v *= inv;
            if (!live) continue;
            if (whole) store_out<QT>(a.out, at, 16 * i + 4 * g, a.c.d, v);
            else *reinterpret_cast<f32x4*>(part + (i * kWave + lane) * 4) = v;
        }
        if (!whole && wave == 0 && g == 0)
            *reinterpret_cast<float2*>(part + 2 * NB * 256 + 2 * col) = make_float2(m, sum);
        if (!whole && t0 == 0 && threadIdx.x == 0) {
            // pieces: this one and those of the workgroups up to the one that has the unit's last tile
            const int64_t rest = s.tiles - t1;
            a.meta[blockIdx.x] = make_int4(b, unit, (int32_t)(1 + (rest + run - 1) / run), 0);
        }
        __syncthreads();
        pos += t1 - t0;
        t0 = 0;
        ++unit;
    }
}

// The pieces of the unit that workgroup blockIdx.x of the first launch started, joined; 16 features (blockIdx.y).
template <int QT>
__global__ void __launch_bounds__(kAttendThreads) attend_join_kernel(AttendArgs a)
{
    __shared__ f32x4 so[kAttendWaves][kWave];
    __shared__ float2 sml[kAttendWaves][kQueries];
    const int4 u = a.meta[blockIdx.x];
    if (u.z == 0) return;
    const int lane = (int)threadIdx.x & (kWave - 1), wave = (int)threadIdx.x / kWave;
    const int col = lane & 15, g = lane >> 4, i = (int)blockIdx.y;
    const int size = part_floats(a.c.nb);
    const Seq s = get_seq(a, u.x, kQueries);
    const int32_t h = u.y / s.blocks, block = u.y - h * s.blocks;
    const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row = (uint32_t)block * kQueries + col;
    const bool live = row < rows;
    float m = -__builtin_inff(), sum = 0.0f;
    f32x4 v = {0, 0, 0, 0};
    for (int k = wave; k < u.z; k += kAttendWaves) {
        const float* part = a.part + (int64_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * size;
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

template <int FMT>
snack_status launch_attend(const AttendArgs& a, int q_fmt, unsigned groups, hipStream_t s)
{
    auto go = [&](auto nb) {
        constexpr int NB = decltype(nb)::value;
        if (q_fmt == SNACK_F32)
            hipLaunchKernelGGL((attend_kernel<FMT, NB, SNACK_F32>), dim3(groups), dim3(kAttendThreads), 0, s, a);
        else
            hipLaunchKernelGGL((attend_kernel<FMT, NB, SNACK_BF16>), dim3(groups), dim3(kAttendThreads), 0, s, a);
    };
    switch (a.c.nb) {
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 3: go(std::integral_constant<int, 3>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 6: go(std::integral_constant<int, 6>{}); break;
    default: go(std::integral_constant<int, 8>{}); break;
    }
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}
// one file a format: attend_int8.hip, attend_e4m3.hip, attend_e2m1.hip
extern template snack_status launch_attend<SNACK_INT8>(const AttendArgs&, int, unsigned, hipStream_t);
extern template snack_status launch_attend<SNACK_E4M3>(const AttendArgs&, int, unsigned, hipStream_t);
extern template snack_status launch_attend<SNACK_E2M1>(const AttendArgs&, int, unsigned, hipStream_t);

}  // namespace snack
