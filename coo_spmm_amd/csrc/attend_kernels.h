// attend_kernels.h -- the two attention kernels: up to 16 queries of a cache head (attend.h says how), and many.
#pragma once

#include "attend.h"

namespace snack {

template <int FMT, int NB, int QT>
__global__ void __launch_bounds__(kAttendThreads, NB <= 4 ? 2 : 1) attend_kernel(AttendArgs a)
{
    constexpr int QP = QT == SNACK_F32 ? 3 : 1, PP = QT == SNACK_F32 ? 3 : 2;
    using Q = typename QType<QT>::T;
    __shared__ Schedule<kAttendThreads> sched;
    __shared__ f32x4 so[kAttendWaves][2 * NB][kWave];
    __shared__ float2 sml[kAttendWaves][kQueries];
    const int lane = (int)threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int col = lane & 15, g = lane >> 4;

    int32_t all_blocks;
    const int64_t total = count_work<kAttendThreads, kQueries>(a, sched, &all_blocks);
    int64_t run = (total + gridDim.x - 1) / gridDim.x;
    if (run < kMinRun) run = kMinRun;
    int64_t pos = run * blockIdx.x;
    const int64_t end = min(total, pos + run);
    if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (pos >= end) return;
    int64_t before;
    Cursor c = find_work<kAttendThreads, kQueries>(a, sched, all_blocks, pos, &before);
    int32_t h = (int32_t)((pos - before) / c.tiles);
    int32_t t0 = (int32_t)(pos - before - (int64_t)h * c.tiles);

    while (pos < end) {
        const Seq s = c.s;
        const int32_t b = c.b, t1 = (int32_t)min((int64_t)c.tiles, t0 + (end - pos));
        const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row0 = (uint32_t)c.k * kQueries;
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
                const int64_t left = bad ? 0 : (int64_t)s.len - base - 8 * g;
                const uint64_t m = first_bytes(left > 8 ? 8 : left < 0 ? 0 : (int)left);
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
        const bool whole = t0 == 0 && t1 == c.tiles;
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
            const int64_t rest = c.tiles - t1;
            a.meta[blockIdx.x] = make_int4(b, c.k, h, (int32_t)(1 + (rest + run - 1) / run));
        }
        __syncthreads();
        pos += t1 - t0;
        t0 = 0;
        if (++h == a.c.heads) {
            h = 0;
            if (pos < end) next_block<kQueries>(a, c);
        }
    }
}

// Many queries of a cache head: 64 NT of them a workgroup, 16 NT a wavefront.  What bounds it is the rate of the
// matrix instructions and of the exponentials beside them, so a tile is decoded once for all four wavefronts: two take
// the halves of K, two the blocks of V, and leave operands in LDS, in the order in which lanes read them (16 bytes a
// lane in a row: no bank conflicts).  Two buffers: while one tile is multiplied, the next is decoded and the one after
// it is on its way from memory, with one barrier a tile.  bf16 queries: probabilities are rounded to bf16 once, which
// the output's own rounding hides (each is off by at most 2^-8 of itself, at random).
template <int FMT, int NB>
struct Share {
    using R = RawTile<FMT, NB>;
    static constexpr int VB = (NB + 1) / 2;   // V blocks of a wavefront
    static constexpr int W = NB * R::KW > VB * R::VW ? NB * R::KW : VB * R::VW;
    static constexpr int E = R::KE > 2 * VB ? R::KE : 2 * VB;
    uint32_t w[W];
    uint32_t e[E];
};
template <int FMT, int NB>
__device__ inline void load_share(Share<FMT, NB>& r, const uint8_t* tile, int role, int lane)
{
    using R = RawTile<FMT, NB>;
    const uint8_t* e = tile + 2 * code_bytes(FMT, NB);
    constexpr int eb = k_exp_bytes(NB);
    if (role < 2) {
        load_chunks<NB, R::KW>(r.w, tile + role * (code_bytes(FMT, NB) / 2), lane);
        const uint8_t* p = e + (16 * role + (lane & 15)) * eb;
        if constexpr (eb == 1) r.e[0] = *p;
        else if constexpr (eb == 2) r.e[0] = *reinterpret_cast<const uint16_t*>(p);
        else load_words<R::KE>(r.e, p);
    } else {
        const uint8_t* v = tile + code_bytes(FMT, NB);
        const uint8_t* ev = e + kTile * eb + (lane >> 4) * NB * 8;
#pragma unroll
        for (int i = 0; i < Share<FMT, NB>::VB; ++i) {
            const int b = 2 * i + role - 2;
            if (b >= NB) break;
            load_words<R::VW>(r.w + i * R::VW, v + v_code_at(FMT, NB, (lane >> 4) * 8, b, lane & 15));
            load_words<2>(r.e + 2 * i, ev + 8 * b);
        }
    }
}

template <int FMT, int NB, int QT, int NT>
__global__ void __launch_bounds__(kAttendThreads, NB * NT <= 8 ? 2 : 1) attend_many_kernel(AttendArgs a)
{
    constexpr int ROWS = 64 * NT;
    constexpr int QP = QT == SNACK_F32 ? 3 : 1, PP = QT == SNACK_F32 ? 3 : 1;
    using Q = typename QType<QT>::T;
    __shared__ Schedule<kAttendThreads> sched;
    __shared__ u32x4 frag[2][4 * NB][kWave];     // K operands of both halves, then V's
    __shared__ uint32_t nans[2][NB];             // tokens of a boundary tile whose block of V is NaN
    const int lane = (int)threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int col = lane & 15, g = lane >> 4;

    int32_t all_blocks;
    const int64_t total = count_work<kAttendThreads, ROWS>(a, sched, &all_blocks);
    int64_t run = (total + gridDim.x - 1) / gridDim.x;
    if (run < kMinRun) run = kMinRun;
    int64_t pos = run * blockIdx.x;
    const int64_t end = min(total, pos + run);
    if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (pos >= end) return;
    int64_t before;
    Cursor c = find_work<kAttendThreads, ROWS>(a, sched, all_blocks, pos, &before);
    int32_t h = (int32_t)((pos - before) / c.tiles);
    int32_t t0 = (int32_t)(pos - before - (int64_t)h * c.tiles);

    while (pos < end) {
        const Seq s = c.s;
        const int32_t b = c.b, t1 = (int32_t)min((int64_t)c.tiles, t0 + (end - pos));
        const uint32_t rows = (uint32_t)s.nq * a.by_group.d, row0 = (uint32_t)c.k * ROWS;
        const int64_t past = a.causal ? (int64_t)s.len - s.nq : (int64_t)s.len - 1;
        // wavefront w has the groups of 16 queries w, w + 4: a block of few queries is still shared out
        uint32_t row[NT];
        int64_t limit[NT];
        bf16x8 q[NT][QP][NB];
        f32x4 o[NT][2 * NB];
        float mc[NT], l[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            row[n] = row0 + 16 * (wave + 4 * n) + col;
            const Row mine = get_row(a, h, min(row[n], rows - 1));
            limit[n] = a.causal ? past + mine.i : past;
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
                for (int k = 0; k < QP; ++k) q[n][k][j] = part[k];
            });
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) o[n][i] = f32x4{0, 0, 0, 0};
            mc[n] = -__builtin_inff();
            l[n] = 0.0f;
        }
        // the last token that the wavefront's first and last query see, and the block's first
        const uint32_t w0 = min(row0 + 16 * wave, rows - 1), w1 = min(row0 + 16 * (wave + 4 * (NT - 1)) + 15, rows - 1);
        const int64_t least = a.causal ? past + fast_quot(a.by_group, w0) : past;
        const int64_t most = row0 + 16 * wave >= rows ? -1 : a.causal ? past + fast_quot(a.by_group, w1) : past;
        const int64_t least_all = a.causal ? past + fast_quot(a.by_group, row0) : past;

        const int32_t* pages = a.table + (int64_t)b * a.width;
        auto page_of = [&](int32_t t) {
            const int32_t p = (int32_t)fast_quot(a.c.by_page, (uint32_t)t);
            return p < a.width ? pages[p] : -1;
        };
        auto is_bad = [&](int32_t page) { return page < 0 || page >= a.pages; };
        Share<FMT, NB> raw;
        auto load = [&](int32_t t, int32_t page) {
            const uint32_t p = fast_quot(a.c.by_page, (uint32_t)t);
            load_share(raw, a.c.data + (int64_t)(is_bad(page) ? 0 : page) * a.c.page_bytes +
                                ((int64_t)h * a.c.page_tiles + (t - p * a.c.page_tiles)) * a.c.record, wave, lane);
        };
        auto stage = [&](int32_t t, int32_t page, int buf) {
            if (wave < 2) {
                unroll<NB>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    frag[buf][wave * NB + j][lane] = __builtin_bit_cast(u32x4, key_operand<FMT, NB, j>(raw.w, raw.e));
                });
                return;
            }
            const int64_t base = (int64_t)t * kTile;
            const bool edge = is_bad(page) || base + kTile - 1 > least_all;
            if (edge) {
                const int64_t left = is_bad(page) ? 0 : (int64_t)s.len - base - 8 * g;
                const uint64_t m = first_bytes(left > 8 ? 8 : left < 0 ? 0 : (int)left);
                unroll<Share<FMT, NB>::VB>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    const int blk = 2 * i + wave - 2;
                    if (blk < NB) {
                        clear_block<FMT>(raw.w + i * RawTile<FMT, NB>::VW, raw.e + 2 * i, m);
                        // what is NaN must not reach a query that does not see it, not even times 0
                        const uint32_t mask = a.causal ? take_nans(raw.e + 2 * i) : 0;
                        if (lane == 0) nans[buf][blk] = mask;
                    }
                });
            }
            unroll<Share<FMT, NB>::VB>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                const int blk = 2 * i + wave - 2;
                if (blk < NB) {
                    bf16x8 lo, hi;
                    value_operands<FMT, NB, i>(raw.w, raw.e, lo, hi);
                    frag[buf][2 * NB + 2 * blk][lane] = __builtin_bit_cast(u32x4, lo);
                    frag[buf][2 * NB + 2 * blk + 1][lane] = __builtin_bit_cast(u32x4, hi);
                }
            });
        };
        int32_t page = page_of(t0), page1 = page_of(min(t0 + 1, t1 - 1));
        load(t0, page);
        stage(t0, page, 0);
        load(min(t0 + 1, t1 - 1), page1);
        __syncthreads();
        for (int32_t t = t0; t < t1; ++t) {
            const int buf = (t - t0) & 1;
            const int32_t page2 = page_of(min(t + 2, t1 - 1));
            if (t + 1 < t1) stage(t + 1, page1, buf ^ 1);
            load(min(t + 2, t1 - 1), page2);
            const int64_t base = (int64_t)t * kTile;
            if (base <= most) {
                f32x4 sc[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const bf16x8 k = __builtin_bit_cast(bf16x8, frag[buf][half * NB + j][lane]);
#pragma unroll
                        for (int i = QP - 1; i >= 0; --i)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                sc[n][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][i][j], sc[n][half], 0, 0, 0);
                    }
                const bool bad = is_bad(page), edge = bad || base + kTile - 1 > least;
                bf16x8 p[NT][PP];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = sc[n][i >> 2][i & 3];
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (bad) x[i] = __builtin_nanf("");
                            if (base + 8 * g + i > limit[n]) x[i] = -__builtin_inff();
                        }
                    }
                    const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                                            fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * a.scale_log2;
                    if (__ballot(top > mc[n] + kRaise)) {
                        const float m = fmaxf(mc[n], query_max(top));
                        const float f = m == mc[n] ? 1.0f : __builtin_amdgcn_exp2f(mc[n] - m);
#pragma unroll
                        for (int i = 0; i < 2 * NB; ++i) o[n][i] *= f;
                        l[n] *= f;
                        mc[n] = m;
                    }
                    const float off = mc[n] == -__builtin_inff() ? 0.0f : -mc[n];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], a.scale_log2, off));
                        l[n] += x[i];
                    }
                    split8<PP>(x, p[n]);
                }
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    const bf16x8 v = __builtin_bit_cast(bf16x8, frag[buf][2 * NB + i][lane]);
#pragma unroll
                    for (int k = PP - 1; k >= 0; --k)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[n][k], o[n][i], 0, 0, 0);
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
            page = page1;
            page1 = page2;
        }

        const bool whole = t0 == 0 && t1 == c.tiles;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float sum = query_sum(l[n]);
            const bool live = row[n] < rows;
            if (whole) {
                const Row mine = get_row(a, h, min(row[n], rows - 1));
                const int64_t at = ((int64_t)(s.first + mine.i) * a.hq + mine.head) * a.c.d;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (live)
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) store_out<QT>(a.out, at, 16 * i + 4 * g, a.c.d, o[n][i] * inv);
            } else if (live) {
                float* part = a.part + ((int64_t)(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * (ROWS / 16) + wave + 4 * n) *
                                           part_floats(NB);
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) *reinterpret_cast<f32x4*>(part + (i * kWave + lane) * 4) = o[n][i];
                if (g == 0) *reinterpret_cast<float2*>(part + 2 * NB * 256 + 2 * col) = make_float2(mc[n], sum);
            }
        }
        if (!whole && t0 == 0 && threadIdx.x == 0) {
            const int64_t rest = c.tiles - t1;
            a.meta[blockIdx.x] = make_int4(b, c.k, h, (int32_t)(1 + (rest + run - 1) / run));
        }
        pos += t1 - t0;
        t0 = 0;
        if (++h == a.c.heads) {
            h = 0;
            if (pos < end) next_block<ROWS>(a, c);
        }
    }
}

template <int FMT>
snack_status launch_attend(const AttendArgs& a, int q_fmt, int kind, unsigned groups, hipStream_t s)
{
    auto go = [&](auto nb, auto qt) {
        constexpr int NB = decltype(nb)::value, QT = decltype(qt)::value;
        // (128 queries of heads past 128 features would not fit the registers: attend_kind)
        const auto k = kind == kFew ? attend_kernel<FMT, NB, QT>
                       : kind == kMany64 ? attend_many_kernel<FMT, NB, QT, 1> : attend_many_kernel<FMT, NB, QT, NB <= 4 ? 2 : 1>;
        hipLaunchKernelGGL(k, dim3(groups), dim3(kAttendThreads), 0, s, a);
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
