// attend_kernels.h -- the two attention kernels: up to 16 queries of a cache head (attend.h says how), and many.
#pragma once

#include "attend.h"

namespace snack {

template <int FMT, int NB, int QT>
__global__ void __launch_bounds__(kAttendThreads, NB <= 4 ? 2 : 1) attend_kernel(AttendArgs a)
{
    constexpr int QP = QT == SNACK_F32 ? 3 : 1, PP = QT == SNACK_F32 ? 3 : 2;
    constexpr int DEPTH = 2;     // tiles of a wavefront in registers: the one in use, one on its way (three: 51 against 48 us
                                 // for 64 streams of up to 4096 tokens, whose last tile is then loaded once more)
    using Q = typename QType<QT>::T;
    __shared__ Schedule<kAttendThreads> sched;
    __shared__ f32x4 so[kAttendWaves][2 * NB][kWave];
    __shared__ float2 sml[kAttendWaves][kQueries];
    const int lane = (int)threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int col = lane & 15, g = lane >> 4;

    int32_t all_blocks;
    const int64_t total = count_work<kAttendThreads, kQueries>(a, sched, &all_blocks);
    int64_t run = divide(total + gridDim.x - 1, gridDim.x);
    if (run < kMinRun) run = kMinRun;
    int64_t pos = run * blockIdx.x;
    const int64_t end = min(total, pos + run);
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) a.meta[a.meta_last] = make_int4(all_blocks * a.c.heads, 0, 0, 0);
        if (!a.by_unit) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    if (pos >= end) return;
    int64_t before;
    int32_t index;
    Cursor c = find_work<kAttendThreads, kQueries>(a, sched, all_blocks, pos, &before, &index);
    int32_t h = (int32_t)divide(pos - before, c.cost);
    int32_t o0 = (int32_t)(pos - before - (int64_t)h * c.cost);     // within the unit

    while (pos < end) {
        const Seq s = c.s;
        const int32_t b = c.b, o1 = (int32_t)min((int64_t)c.cost, o0 + (end - pos));
        const int32_t t0 = max(o0 - unit_cost<kQueries>(), 0), t1 = max(o1 - unit_cost<kQueries>(), 0);
        if (t1 == 0) break;      // the next workgroup starts it
        const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row0 = (uint32_t)c.k * kQueries;
        const uint32_t row = row0 + col;
        const bool live = row < rows;
        const Row mine = get_row(a, h, live ? row : rows - 1);
        // the last token a query sees, of this lane's and of the unit's first
        const int64_t past = a.causal ? (int64_t)s.len - s.nq : (int64_t)s.len - 1;
        const int64_t limit = a.causal ? past + mine.i : past;
        const int64_t least = a.causal ? past + fast_quot(a.by_group, row0) : past;

        f32x4 o[2 * NB];
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) o[i] = f32x4{0, 0, 0, 0};
        float mc = -__builtin_inff(), l = 0.0f;   // running maximum times scale_log2; this lane's sum

        const Fixed<int32_t> pages = fixed(a.table) + (int64_t)b * a.width;
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
        // tiles t0 + wave, + 4, ... up to t1; the last again where there is none
        auto at_most = [&](int32_t t) { return min(t, t1 - 1); };
        auto is_bad = [&](int32_t p) { return p < 0 || p >= a.pages; };
        RawTile<FMT, NB> raw[DEPTH];
        uint32_t bad_tiles = 0;      // bit i: the i-th tile from the present one on has no page
        int32_t page;
        {
            int32_t p[DEPTH];
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) p[i] = page_of(at_most(t0 + wave + kAttendWaves * i));
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                load_tile(raw[i], tile_at(at_most(t0 + wave + kAttendWaves * i), p[i]), lane);
                bad_tiles |= is_bad(p[i]) ? 1u << i : 0u;
                // in this order: what is waited for in the loop is counted in loads behind it, by both ways into it
                __builtin_amdgcn_sched_barrier(0);
            }
            page = page_of(at_most(t0 + wave + kAttendWaves * DEPTH));
        }
        bf16x8 q[QP][NB];
        {
            f32x8 x[NB];
            load_query<NB>(x, (const Q*)a.q + (int64_t)(s.first + mine.i) * a.q_row + (int64_t)mine.head * a.q_head, 8 * g, a.c.d);
            split_query<QP, NB>(q, x);
        }
        auto multiply = [&](int32_t t, RawTile<FMT, NB>& cur) {
            const int64_t base = (int64_t)t * kTile;
            const bool bad = bad_tiles & 1u;
            f32x4 sc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
            unroll<NB>([&](auto jc) {
                constexpr int j = decltype(jc)::value;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const bf16x8 k = key_operand<FMT, j % 4>(cur.k[half] + j * RawTile<FMT, NB>::KW, cur.ke[half][j / 4]);
#pragma unroll
                    for (int i = QP - 1; i >= 0; --i)
                        sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[i][j], sc[half], 0, 0, 0);
                }
            });
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][i & 3];
            if (bad || base + kTile - 1 > least) {
                const uint64_t m = bad ? 0 : first_bytes(tokens_seen((int64_t)s.len - 1, base, g));
                unroll<NB>([&](auto bc) {
                    constexpr int blk = decltype(bc)::value;
                    clear_block<FMT>(cur.v + blk * RawTile<FMT, NB>::VW, cur.ve + 2 * blk, m);
                    // what is NaN must not reach a query that does not see it, not even times 0
                    uint32_t tokens = a.causal ? take_nans(cur.ve + 2 * blk) : 0;
                    while (tokens) {
                        const int tok = __ffs(tokens) - 1;
                        tokens &= tokens - 1;
                        if (base + tok <= limit) {
                            const float nan = __builtin_nanf("");
                            o[2 * blk] = o[2 * blk + 1] = f32x4{nan, nan, nan, nan};
                        }
                    }
                });
                if (bad)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
                const int seen = tokens_seen(limit, base, g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= seen) x[i] = -__builtin_inff();
            }
            const float top = max8(x) * a.scale_log2;
            if (__ballot(top > mc + kRaise)) {
                const float m = raised(mc, query_max(top));
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
                value_operands<FMT>(cur.v + blk * RawTile<FMT, NB>::VW, cur.ve + 2 * blk, lo, hi);
#pragma unroll
                for (int i = PP - 1; i >= 0; --i) {
                    o[2 * blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, p[i], o[2 * blk], 0, 0, 0);
                    o[2 * blk + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, p[i], o[2 * blk + 1], 0, 0, 0);
                }
            });
        };
        // The same registers for a tile each time round (a copy would wait for it), and one way out of the loop.
        for (int32_t t = t0 + wave; t < t1; t += kAttendWaves * DEPTH)
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const int32_t at = t + kAttendWaves * i;
                if (at < t1) multiply(at, raw[i]);
                load_tile(raw[i], tile_at(at_most(at + kAttendWaves * DEPTH), page), lane);
                bad_tiles = bad_tiles >> 1 | (is_bad(page) ? 1u << (DEPTH - 1) : 0u);
                page = page_of(at_most(at + kAttendWaves * (DEPTH + 1)));
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
        const bool whole = t0 == 0 && t1 == c.tiles;
        float* part = a.part + (int64_t)(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * part_floats(NB);
        const int64_t at = ((int64_t)(s.first + mine.i) * a.hq + mine.head) * a.c.d;
        const float inv = whole ? inverse_sum(sum, limit) : 1.0f;
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
        if (t0 == 0 && threadIdx.x == 0 && (a.by_unit || !whole)) {
            // pieces: this one and those of the workgroups up to the one that has the unit's last tile
            const int64_t rest = c.cost - o1;
            int4* m = a.meta + 2 * (a.by_unit ? index * a.c.heads + h : (int32_t)blockIdx.x);
            m[0] = make_int4(s.first, c.k, h, whole ? 0 : (int32_t)(1 + divide(rest + run - 1, run)));
            m[1] = make_int4((int32_t)rows, (int32_t)blockIdx.x, (int32_t)past, 0);
        }
        __syncthreads();
        pos += o1 - o0;
        o0 = 0;
        if (++h == a.c.heads) {
            h = 0;
            ++index;
            if (pos < end) next_block<kQueries>(a, c);
        }
    }
}

// Many queries of a cache head: 16 NT of them a wavefront, W wavefronts.  What bounds it is the issue of the matrix
// instructions and of the exponentials and conversions beside them, so a tile is decoded once for all wavefronts: half
// of them take a share of K, half one of V, and leave operands in LDS, in the order in which lanes read them (16
// bytes a lane in a row: no bank conflicts).  Two buffers: while one tile is multiplied, the next is decoded and the
// one after it is on its way from memory, with one barrier a tile.  bf16 queries: a probability is the sum of two bf16
// numbers, off by at most 2^-16 of itself, as in the kernel of few queries, so that a query's result does not depend on
// which kernel the call's other sequences put it into; the sum of the probabilities is one more row of the second
// product.  (512 queries over 8192 tokens: 132 us, with one bf16 number 109; but where values cancel that one's error is as
// large as the output's own rounding, and the error against 64 bits 2.2e-3 against 1.7e-3.)
//
// A share is units of the words of one V block, or of two neighbouring blocks of one half of K, which are as many:
// wavefront w of the first half has half w % 2 and the units w / 2, w / 2 + W / 4, ..., one of the second the V blocks
// w - W / 2, w, ...  So every wavefront has the same loads, from places of its own: a branch round them would bring
// their registers together behind it, and wait for them there.
template <int FMT, int NB, int W>
struct Share {
    using R = RawTile<FMT, NB>;
    static constexpr int UNITS = (NB + W / 2 - 1) / (W / 2);
    uint32_t w[UNITS][R::VW];
    uint32_t e[UNITS][2];
};
template <int FMT, int NB, int W>
struct Places {
    static constexpr int UNITS = Share<FMT, NB, W>::UNITS;
    uint32_t w[UNITS], e[UNITS];   // this lane's bytes in a tile
    uint32_t shift[UNITS];         // K: where its exponents start in the words
};
// unit i of a wavefront: K's first block, V's block (NB and more: none)
template <int W>
__device__ inline int unit_block(int wave, int i)
{
    return wave < W / 2 ? 2 * ((wave >> 1) + W / 4 * i) : wave - W / 2 + W / 2 * i;
}
template <int FMT, int NB, int W>
__device__ inline void find_places(Places<FMT, NB, W>& p, int wave, int lane)
{
    constexpr int eb = k_exp_bytes(NB);
#pragma unroll
    for (int i = 0; i < Places<FMT, NB, W>::UNITS; ++i) {
        const int b = min(unit_block<W>(wave, i), wave < W / 2 ? (NB - 1) / 2 * 2 : NB - 1);
        if (wave < W / 2) {
            const int t = 8 * ((lane & 15) >> 2) + 4 * (wave & 1) + (lane & 3);
            p.w[i] = k_code_at(FMT, NB, t, b, lane >> 4);
            const uint32_t at = k_exp_at(NB, t, b);
            p.e[i] = 2 * code_bytes(FMT, NB) + (at & ~3u);
            p.shift[i] = 8 * (at & 3u);
        } else {
            p.w[i] = code_bytes(FMT, NB) + v_code_at(FMT, NB, (lane >> 4) * 8, b, lane & 15);
            p.e[i] = 2 * code_bytes(FMT, NB) + kTile * eb + v_exp_at(NB, (lane >> 4) * 8, b);
            p.shift[i] = 0;
        }
    }
}
template <int FMT, int NB, int W>
__device__ inline void load_share(Share<FMT, NB, W>& r, const uint8_t* tile, const Places<FMT, NB, W>& p)
{
#pragma unroll
    for (int i = 0; i < Share<FMT, NB, W>::UNITS; ++i) {
        load_words<RawTile<FMT, NB>::VW>(r.w[i], tile + p.w[i]);
        load_words<2>(r.e[i], tile + p.e[i]);
    }
}

template <int FMT, int NB, int QT, int W, int NT>
__global__ void __launch_bounds__(W * kWave, NB * NT <= 8 ? 2 : 1) attend_many_kernel(AttendArgs a)
{
    constexpr int THREADS = W * kWave, ROWS = 16 * W * NT;
    constexpr int QP = QT == SNACK_F32 ? 3 : 1, PP = QT == SNACK_F32 ? 3 : 2;
    constexpr bool kSumRow = QT != SNACK_F32;
    using Q = typename QType<QT>::T;
    using S = Share<FMT, NB, W>;
    constexpr int DEPTH = 2;     // tiles on their way from memory
    __shared__ Schedule<THREADS> sched;
    __shared__ u32x4 kfrag[2][2 * NB][kWave], vfrag[2][2 * NB][kWave];   // K operands of both halves; V's
    __shared__ uint32_t nans[2][NB];             // tokens of a boundary tile whose block of V is NaN
    const int lane = (int)threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int col = lane & 15, g = lane >> 4;
    const bool keys = wave < W / 2;
    Places<FMT, NB, W> places;
    find_places(places, wave, lane);

    int32_t all_blocks;
    const int64_t total = count_work<THREADS, ROWS>(a, sched, &all_blocks);
    int64_t run = divide(total + gridDim.x - 1, gridDim.x);
    if (run < kMinRun) run = kMinRun;
    int64_t pos = run * blockIdx.x;
    const int64_t end = min(total, pos + run);
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) a.meta[a.meta_last] = make_int4(all_blocks * a.c.heads, 0, 0, 0);
        if (!a.by_unit) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    if (pos >= end) return;
    int64_t before;
    int32_t index;
    Cursor c = find_work<THREADS, ROWS>(a, sched, all_blocks, pos, &before, &index);
    int32_t h = (int32_t)divide(pos - before, c.cost);
    int32_t o0 = (int32_t)(pos - before - (int64_t)h * c.cost);     // within the unit

    while (pos < end) {
        const Seq s = c.s;
        const int32_t b = c.b, o1 = (int32_t)min((int64_t)c.cost, o0 + (end - pos));
        const int32_t t0 = max(o0 - unit_cost<ROWS>(), 0), t1 = max(o1 - unit_cost<ROWS>(), 0);
        if (t1 == 0) break;      // the next workgroup starts it
        const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row0 = (uint32_t)c.k * ROWS;
        const int64_t past = a.causal ? (int64_t)s.len - s.nq : (int64_t)s.len - 1;
        // wavefront w has the groups of 16 queries w, w + W: a block of few queries is still shared out
        uint32_t row[NT];
        int64_t limit[NT];
        const Q* query[NT];
        bf16x8 q[NT][QP][NB];
        f32x4 o[NT][2 * NB];
        float mc[NT], l[NT];     // running maximum times scale_log2; this lane's sum
        f32x4 lsum[NT];          // the sum over all lanes, where the product makes it
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            row[n] = row0 + 16 * (wave + W * n) + col;
            const Row mine = get_row(a, h, min(row[n], rows - 1));
            limit[n] = a.causal ? past + mine.i : past;
            query[n] = (const Q*)a.q + (int64_t)(s.first + mine.i) * a.q_row + (int64_t)mine.head * a.q_head;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) o[n][i] = f32x4{0, 0, 0, 0};
            mc[n] = -__builtin_inff();
            l[n] = 0.0f;
            lsum[n] = f32x4{0, 0, 0, 0};
        }
        // the last token that the wavefront's first and last query see, and the block's first
        const uint32_t w0 = min(row0 + 16 * wave, rows - 1), w1 = min(row0 + 16 * (wave + W * (NT - 1)) + 15, rows - 1);
        const int64_t least = a.causal ? past + fast_quot(a.by_group, w0) : past;
        const int64_t most = row0 + 16 * wave >= rows ? -1 : a.causal ? past + fast_quot(a.by_group, w1) : past;
        const int64_t least_all = a.causal ? past + fast_quot(a.by_group, row0) : past;

        const Fixed<int32_t> pages = fixed(a.table) + (int64_t)b * a.width;
        auto page_of = [&](int32_t t) {
            const int32_t p = (int32_t)fast_quot(a.c.by_page, (uint32_t)t);
            return p < a.width ? pages[p] : -1;
        };
        auto is_bad = [&](int32_t page) { return page < 0 || page >= a.pages; };
        auto load = [&](S& raw, int32_t t, int32_t page) {
            const uint32_t p = fast_quot(a.c.by_page, (uint32_t)t);
            load_share(raw, a.c.data + (int64_t)(is_bad(page) ? 0 : page) * a.c.page_bytes +
                                ((int64_t)h * a.c.page_tiles + (t - p * a.c.page_tiles)) * a.c.record, places);
        };
        // the wavefront's share of tile t becomes operands
        auto stage = [&](S& raw, int32_t t, bool bad, int buf) {
            if (keys) {
                unroll<S::UNITS>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    const int blk = unit_block<W>(wave, i);
                    const uint32_t e = raw.e[i][0] >> places.shift[i];
                    u32x4* to = &kfrag[buf][(wave & 1) * NB + blk][lane];
                    if (blk < NB) to[0] = __builtin_bit_cast(u32x4, key_operand<FMT, 0>(raw.w[i], e));
                    if (blk + 1 < NB)
                        to[kWave] = __builtin_bit_cast(u32x4, key_operand<FMT, 1>(raw.w[i] + RawTile<FMT, NB>::KW, e));
                });
                return;
            }
            const int64_t base = (int64_t)t * kTile;
            if (bad || base + kTile - 1 > least_all) {
                const uint64_t m = bad ? 0 : first_bytes(tokens_seen((int64_t)s.len - 1, base, g));
                unroll<S::UNITS>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    const int blk = unit_block<W>(wave, i);
                    clear_block<FMT>(raw.w[i], raw.e[i], m);
                    // what is NaN must not reach a query that does not see it, not even times 0
                    const uint32_t mask = a.causal ? take_nans(raw.e[i]) : 0;
                    if (lane == 0 && blk < NB) nans[buf][blk] = mask;
                });
            }
            unroll<S::UNITS>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                const int blk = unit_block<W>(wave, i);
                if (blk < NB) {
                    bf16x8 lo, hi;
                    value_operands<FMT>(raw.w[i], raw.e[i], lo, hi);
                    vfrag[buf][2 * blk][lane] = __builtin_bit_cast(u32x4, lo);
                    vfrag[buf][2 * blk + 1][lane] = __builtin_bit_cast(u32x4, hi);
                }
            });
        };
        const uint32_t one2 = 0x3F803F80u;
        const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{one2, one2, one2, one2});
        // the operands that a buffer holds, and the scores from K's
        auto read_operands = [&](bf16x8(&f)[2 * NB], const u32x4(*from)[kWave]) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) f[i] = __builtin_bit_cast(bf16x8, from[i][lane]);
        };
        auto scores = [&](f32x4(&sc)[NT][2], const bf16x8(&k)[2 * NB]) {
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = QP - 1; i >= 0; --i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            sc[n][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[half * NB + j], q[n][i][j], sc[n][half], 0, 0, 0);
        };
        auto largest = [&](const f32x4* sc) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][i & 3];
            return max8(x) * a.scale_log2;
        };
        auto at_most = [&](int32_t t) { return min(t, t1 - 1); };
        // Tile t's probabilities and second product go side by side with the first product of tile t + 1: K runs one
        // tile ahead of V.  Behind what is staged, DEPTH tiles are on their way: one takes 1.3 us under load, about
        // the time of a tile's products.
        const int ahead = keys ? 2 : 1;
        S raw[DEPTH];
        uint32_t bad_tiles = 0;    // bit i: tile t + i has no page
        {
            S first, second;
            const int32_t p0 = page_of(t0), p1 = page_of(at_most(t0 + 1));
            load(first, t0, p0);
            load(second, at_most(t0 + 1), p1);
            bad_tiles = (is_bad(p0) ? 1u : 0u) | (is_bad(p1) ? 2u : 0u);
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const int32_t p = page_of(at_most(t0 + ahead + i));
                load(raw[i], at_most(t0 + ahead + i), p);
                bad_tiles |= is_bad(p) ? 1u << (ahead + i) : 0u;
                // in this order: what is waited for in the loop is counted in loads behind it, by both ways into it
                __builtin_amdgcn_sched_barrier(0);
            }
            f32x8 x[NT][NB];
#pragma unroll
            for (int n = 0; n < NT; ++n) load_query<NB>(x[n], query[n], 8 * g, a.c.d);
#pragma unroll
            for (int n = 0; n < NT; ++n) split_query<QP, NB>(q[n], x[n]);
            stage(first, t0, bad_tiles & 1u, 0);
            if (keys) stage(second, at_most(t0 + 1), false, 1);
        }
        int32_t page = page_of(at_most(t0 + ahead + DEPTH));
        __syncthreads();
        f32x4 sc[NT][2];
        float top[NT];
        {
            bf16x8 k[2 * NB];
            read_operands(k, kfrag[0]);
            scores(sc, k);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) top[n] = largest(sc[n]);
        __syncthreads();     // the first K operands are read: they make room for the third tile's
        int buf = 0;
        auto step = [&](int32_t t, S& share) {
            stage(share, at_most(t + ahead), bad_tiles >> ahead & 1u, keys ? buf : buf ^ 1);
            load(share, at_most(t + ahead + DEPTH), page);
            bad_tiles |= is_bad(page) ? 1u << (ahead + DEPTH) : 0u;
            page = page_of(at_most(t + ahead + DEPTH + 1));
            const int64_t base = (int64_t)t * kTile;
            if (base <= most && t < t1) {
                const bool bad = bad_tiles & 1u;
                if (bad || base + kTile - 1 > least) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int seen = tokens_seen(limit[n], base, g);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (bad) sc[n][i >> 2][i & 3] = __builtin_nanf("");
                            if (i >= seen) sc[n][i >> 2][i & 3] = -__builtin_inff();
                        }
                        top[n] = largest(sc[n]);
                    }
                }
                float off[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (__ballot(top[n] > mc[n] + kRaise)) {
                        const float m = raised(mc[n], query_max(top[n]));
                        const float f = m == mc[n] ? 1.0f : __builtin_amdgcn_exp2f(mc[n] - m);
#pragma unroll
                        for (int i = 0; i < 2 * NB; ++i) o[n][i] *= f;
                        if constexpr (kSumRow) lsum[n] *= f;
                        else l[n] *= f;
                        mc[n] = m;
                    }
                    off[n] = mc[n] == -__builtin_inff() ? 0.0f : -mc[n];
                }
                bf16x8 k[2 * NB], v[2 * NB];
                read_operands(k, kfrag[buf ^ 1]);
                read_operands(v, vfrag[buf]);
                f32x4 next[NT][2];
                scores(next, k);
                bf16x8 p[NT][PP];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = __builtin_amdgcn_exp2f(fmaf(sc[n][i >> 2][i & 3], a.scale_log2, off[n]));
                        if constexpr (!kSumRow) l[n] += x[i];
                    }
                    split8<PP>(x, p[n]);
                }
                if constexpr (kSumRow) {
#pragma unroll
                    for (int j = PP - 1; j >= 0; --j)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            lsum[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, p[n][j], lsum[n], 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
#pragma unroll
                    for (int j = PP - 1; j >= 0; --j)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[i], p[n][j], o[n][i], 0, 0, 0);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sc[n][0] = next[n][0];
                    sc[n][1] = next[n][1];
                    top[n] = largest(sc[n]);
                }
                // a tile that is an edge for the block's first query: the staging wavefronts took its NaN out
                if (a.causal && (bad || base + kTile - 1 > least_all)) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        uint32_t m = nans[buf][i];
                        while (m) {
                            const int tok = __ffs(m) - 1;
                            m &= m - 1;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                if (base + tok <= limit[n]) {
                                    const float nan = __builtin_nanf("");
                                    o[n][2 * i] = o[n][2 * i + 1] = f32x4{nan, nan, nan, nan};
                                }
                        }
                    }
                }
            }
            __syncthreads();
            bad_tiles >>= 1;
            buf ^= 1;
        };
        // The same registers for a share each time round (a copy would wait for it), and one way out: what a share's
        // use has to wait for is counted in the loads behind it, on every way there.
        for (int32_t t = t0; t < t1; t += DEPTH)
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) step(t + i, raw[i]);

        const bool whole = t0 == 0 && t1 == c.tiles;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float sum = kSumRow ? lsum[n][0] : query_sum(l[n]);
            const bool live = row[n] < rows;
            if (whole) {
                const Row mine = get_row(a, h, min(row[n], rows - 1));
                const int64_t at = ((int64_t)(s.first + mine.i) * a.hq + mine.head) * a.c.d;
                const float inv = inverse_sum(sum, limit[n]);
                if (live)
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) store_out<QT>(a.out, at, 16 * i + 4 * g, a.c.d, o[n][i] * inv);
            } else if (live) {
                float* part = a.part + ((int64_t)(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * (ROWS / 16) + wave + W * n) *
                                           part_floats(NB);
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) *reinterpret_cast<f32x4*>(part + (i * kWave + lane) * 4) = o[n][i];
                if (g == 0) *reinterpret_cast<float2*>(part + 2 * NB * 256 + 2 * col) = make_float2(mc[n], sum);
            }
        }
        if (t0 == 0 && threadIdx.x == 0 && (a.by_unit || !whole)) {
            const int64_t rest = c.cost - o1;
            int4* m = a.meta + 2 * (a.by_unit ? index * a.c.heads + h : (int32_t)blockIdx.x);
            m[0] = make_int4(s.first, c.k, h, whole ? 0 : (int32_t)(1 + divide(rest + run - 1, run)));
            m[1] = make_int4((int32_t)rows, (int32_t)blockIdx.x, (int32_t)past, 0);
        }
        pos += o1 - o0;
        o0 = 0;
        if (++h == a.c.heads) {
            h = 0;
            ++index;
            if (pos < end) next_block<ROWS>(a, c);
        }
    }
}

template <int FMT>
snack_status launch_attend(const AttendArgs& a, int q_fmt, int kind, unsigned groups, hipStream_t s)
{
    auto go = [&](auto nb, auto qt) {
        constexpr int NB = decltype(nb)::value, QT = decltype(qt)::value;
        if (kind == kFew)
            hipLaunchKernelGGL((attend_kernel<FMT, NB, QT>), dim3(groups), dim3(kAttendThreads), 0, s, a);
        else if (kind == kMany64)
            hipLaunchKernelGGL((attend_many_kernel<FMT, NB, QT, 4, 1>), dim3(groups), dim3(4 * kWave), 0, s, a);
        else if constexpr (NB <= 4)
            hipLaunchKernelGGL((attend_many_kernel<FMT, NB, QT, 8, 2>), dim3(groups), dim3(8 * kWave), 0, s, a);
    };
    auto types = [&](auto nb) {
        if (q_fmt == SNACK_F32) go(nb, std::integral_constant<int, SNACK_F32>{});
        else go(nb, std::integral_constant<int, SNACK_BF16>{});
    };
    switch (a.c.nb) {
    case 1: types(std::integral_constant<int, 1>{}); break;
    case 2: types(std::integral_constant<int, 2>{}); break;
    case 3: types(std::integral_constant<int, 3>{}); break;
    case 4: types(std::integral_constant<int, 4>{}); break;
    case 6: types(std::integral_constant<int, 6>{}); break;
    default: types(std::integral_constant<int, 8>{}); break;
    }
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

}  // namespace snack
