// cache.hip -- the pass from the projections' output to the attention (norms and
// rotation of queries and keys, keys and values into the cache), slots, read back.
//
// One launch, one pass over its input, bound by HBM: a head of a token on a group of
// lanes, eight features each.  The norm and the rotation are computed in 64 bits (as
// many operations a cycle as in 32 without packing): a value of a key next to a
// border of the cache's grid then lies on the right side of it.
#include "cache.h"
#include "rope.h"

namespace snack {
namespace {

constexpr int kThreads = 256;
// Workgroups of a launch at most: HIP takes fewer than 2^32 threads.  What needs more is launched in pieces.
constexpr uint32_t kLaunchGroups = 1u << 23;

__device__ inline uint32_t abs_max8(f32x8 x)
{
    return max(abs_max4(f32x4{x[0], x[1], x[2], x[3]}), abs_max4(f32x4{x[4], x[5], x[6], x[7]}));
}
// over the four lanes of a block
__device__ inline uint32_t quad_max(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));
    return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));
}

// eight features of a key, of block b and its eighth-features g, to token t of a tile
template <int FMT>
__device__ inline void store_key(uint8_t* tile, int nb, int t, int b, int g, f32x8 y)
{
    const uint32_t s = cache_exponent<FMT>(quad_max(abs_max8(y)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cache_encode2<FMT>(y[2 * i], y[2 * i + 1], s);
    uint8_t* at = tile + k_code_at(FMT, nb, t, b, g);
    if constexpr (four_bits(FMT)) {
        *reinterpret_cast<uint32_t*>(at) = w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24;
    } else {
        *reinterpret_cast<uint2*>(at) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
    if (g == 0) tile[2 * code_bytes(FMT, nb) + k_exp_at(nb, t, b)] = (uint8_t)s;
}
// Four features of a key, 4 f .. 4 f + 3; the eight lanes of a block are neighbours.
template <int FMT>
__device__ inline void store_key4(uint8_t* tile, int nb, int t, int f, f32x4 y)
{
    const uint32_t s = cache_exponent<FMT>(octet_max(abs_max4(y)));
    const uint32_t lo = cache_encode2<FMT>(y.x, y.y, s), hi = cache_encode2<FMT>(y.z, y.w, s);
    const int b = f >> 3, g = (f & 7) >> 1, second = f & 1;
    uint8_t* at = tile + k_code_at(FMT, nb, t, b, g);
    if constexpr (four_bits(FMT)) reinterpret_cast<uint16_t*>(at)[second] = (uint16_t)(lo | hi << 8);
    else reinterpret_cast<uint32_t*>(at)[second] = lo | hi << 16;
    if ((f & 7) == 0) tile[2 * code_bytes(FMT, nb) + k_exp_at(nb, t, b)] = (uint8_t)s;
}
// features 32 b + 4 g + 0..3 and 32 b + 16 + 4 g + 0..3 of a value
template <int FMT>
__device__ inline void store_value(uint8_t* tile, int nb, int t, int b, int g, f32x8 y)
{
    const uint32_t s = cache_exponent<FMT>(quad_max(abs_max8(y)));
    uint8_t* codes = tile + code_bytes(FMT, nb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = cache_encode2<FMT>(y[i], y[4 + i], s);
        uint8_t* at = codes + v_code_at(FMT, nb, t, b, 4 * g + i);
        if constexpr (four_bits(FMT)) *at = (uint8_t)w;
        else *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
    }
    if (g == 0) tile[2 * code_bytes(FMT, nb) + kTile * k_exp_bytes(nb) + v_exp_at(nb, t, b)] = (uint8_t)s;
}

// four features from p, of which the first `left` exist
template <typename X>
__device__ inline f32x4 part4(const X* p, int left)
{
    f32x4 v = {0, 0, 0, 0};
    if (left >= 4) {
        if constexpr (sizeof(X) == 4) {
            v = *reinterpret_cast<const f32x4u*>(p);
        } else {
            const u16x4u h = *reinterpret_cast<const u16x4u*>(p);
            v = f32x4{bf16_value(h.x), bf16_value(h.y), bf16_value(h.z), bf16_value(h.w)};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) v[i] = load1(p + i);
    }
    return v;
}

// Workgroups 0..gq-1: queries, then gk of keys, then those of values.  Measured: 8192 tokens of 32 query and 8 key heads
// of 128, fp32 to bf16, 254 MB in 59 us (4.3 TB/s); 8192 tokens of 12 heads of 64 into an int8 cache, 114 MB in 44 us (the
// values' codes go out two bytes at a time, into lines that eight tokens fill: 54 MB written for 38); one token 3.0 us
// (a launch).  EVEN spares
// the selects that move a partial four into place: 59 against 84 us.
template <int LPR, bool EVEN, typename X, typename Y>
__global__ void __launch_bounds__(kThreads) qk_pass_kernel(QkPass a, CacheView c, int fmt, uint32_t gq, uint32_t gk, uint32_t first)
{
    uint32_t group = first + blockIdx.x;
    const int kind = group < gq ? 0 : group < gq + gk ? 1 : 2;
    if (kind == 1) group -= gq;
    if (kind == 2) group -= gq + gk;
    const Heads& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int lane = (int)threadIdx.x % LPR, f0 = 8 * lane;
    const uint32_t row = group * (kThreads / LPR) + threadIdx.x / LPR;
    const bool live = row < in.rows;
    // every lane stays: sums and maxima are taken over neighbouring lanes
    const uint32_t rr = live ? row : in.rows - 1;
    const uint32_t token = fast_quot(in.heads, rr), h = rr - token * in.heads.d;
    const X* p = (const X*)in.p + (int64_t)token * in.row + (int64_t)h * in.head;
    const bool kept = kind == 2 || (kind == 1 && !a.yk);
    const int64_t slot = kept ? a.slot[token] : 0;
    const bool place = kept && live && slot >= 0 && slot < c.slots;
    if (kind == 2) {
        const int b = lane >> 2, g = lane & 3, n = 32 * b + 4 * g;
        const f32x4 lo = part4(p + n, a.d - n), hi = part4(p + n + 16, a.d - n - 16);
        const f32x8 y = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        if (!place || b >= c.nb) return;
        uint8_t* tile = cache_tile(c, slot, (int)h);
        const int t = (int)(slot & (kTile - 1));
        if (fmt == SNACK_INT8) store_value<SNACK_INT8>(tile, c.nb, t, b, g, y);
        else if (fmt == SNACK_E4M3) store_value<SNACK_E4M3>(tile, c.nb, t, b, g, y);
        else store_value<SNACK_E2M1>(tile, c.nb, t, b, g, y);
        return;
    }
    // whole pairs on a lane: outputs always, keys for the cache where a block's lanes are then neighbours
    if (!kept || a.key_pairs) {
        const Spot8 at = find_spot8(lane, a.d, a.ro.r, a.ro.layout);
        const Eight z = qk_pairs<LPR, EVEN>(p, at, lane, a.d, kind == 0 ? a.q_gain : a.k_gain, a.eps, a.inv_d, a.ro,
                                      a.ro.table ? a.pos[token] : 0);
        if (!kept) {
            Y* to = (Y*)(kind == 0 ? a.yq : a.yk) + (int64_t)row * a.d;
            if (live) {
                put4(to + at.a, z.a, at.na);
                put4(to + at.b, z.b, at.nb);
            }
            return;
        }
        if (!place || !at.turned) return;
        uint8_t* tile = cache_tile(c, slot, (int)h);
        const int t = (int)(slot & (kTile - 1)), fa = at.a >> 2, fb = at.b >> 2;
        if (fmt == SNACK_INT8) {
            store_key4<SNACK_INT8>(tile, c.nb, t, fa, z.a);
            store_key4<SNACK_INT8>(tile, c.nb, t, fb, z.b);
        } else if (fmt == SNACK_E4M3) {
            store_key4<SNACK_E4M3>(tile, c.nb, t, fa, z.a);
            store_key4<SNACK_E4M3>(tile, c.nb, t, fb, z.b);
        } else {
            store_key4<SNACK_E2M1>(tile, c.nb, t, fa, z.a);
            store_key4<SNACK_E2M1>(tile, c.nb, t, fb, z.b);
        }
        return;
    }
    const f64x8 z = qk_value<LPR>(p, f0, a.d, kind == 0 ? a.q_gain : a.k_gain, a.eps, a.inv_d, a.ro,
                                  a.ro.table ? a.pos[token] : 0);
    const f32x8 y = __builtin_convertvector(z, f32x8);
    const int b = lane >> 2, g = lane & 3;
    if (!place || b >= c.nb) return;
    uint8_t* tile = cache_tile(c, slot, (int)h);
    const int t = (int)(slot & (kTile - 1));
    if (fmt == SNACK_INT8) store_key<SNACK_INT8>(tile, c.nb, t, b, g, y);
    else if (fmt == SNACK_E4M3) store_key<SNACK_E4M3>(tile, c.nb, t, b, g, y);
    else store_key<SNACK_E2M1>(tile, c.nb, t, b, g, y);
}

__global__ void __launch_bounds__(kThreads)
slots_kernel(const int32_t* __restrict__ table, int32_t width, const int32_t* __restrict__ lens,
             const int32_t* __restrict__ starts, int32_t sequences, int32_t per, int32_t tokens, int32_t page_tokens,
             int64_t pages, int32_t* __restrict__ pos, int64_t* __restrict__ slot)
{
    const int32_t i = (int32_t)(blockIdx.x * kThreads + threadIdx.x);
    if (i >= tokens) return;
    int32_t b, first, last;
    if (starts) {
        // the last sequence that starts at or before i
        int32_t lo = 0, hi = sequences;
        while (lo < hi) {
            const int32_t m = (lo + hi) >> 1;
            if (starts[m + 1] > i) hi = m;
            else lo = m + 1;
        }
        b = lo;
        first = b < sequences ? starts[b] : 0;
        last = b < sequences ? starts[b + 1] : 0;
    } else {
        b = i / per;
        first = b * per;
        last = first + per;
    }
    int32_t p = 0;
    int64_t s = -1;
    if (b < sequences && i >= first) {
        const int64_t at = (int64_t)lens[b] - last + i;
        if (at >= 0) {
            p = (int32_t)at;
            const int64_t w = at / page_tokens;
            if (w < width) {
                const int32_t page = table[(int64_t)b * width + w];
                if (page >= 0 && page < pages) s = (int64_t)page * page_tokens + (at - w * page_tokens);
            }
        }
    }
    pos[i] = p;
    slot[i] = s;
}

// Eight features a lane, as they were written.  Token by token, so a tile's lines go to many workgroups and their caches:
// 8192 tokens of 12 heads of 64 from an int8 cache in 16 us, 50 MB fetched for the 13 that are kept.
template <int LPR, int FMT, typename Y>
__global__ void __launch_bounds__(kThreads)
read_kernel(CacheView c, const int64_t* __restrict__ slots, FastDiv heads, uint32_t rows, uint32_t gk, uint32_t first,
            Y* __restrict__ K, Y* __restrict__ V)
{
    const uint32_t at = first + blockIdx.x;
    const bool value = at >= gk;
    const uint32_t group = value ? at - gk : at;
    const int lane = (int)threadIdx.x % LPR;
    const uint32_t row = group * (kThreads / LPR) + threadIdx.x / LPR;
    const int b = lane >> 2, g = lane & 3;
    if (row >= rows || b >= c.nb) return;
    const uint32_t token = fast_quot(heads, row), h = row - token * heads.d;
    const int64_t slot = slots[token];
    f32x8 y = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= c.slots) {
        y += __builtin_nanf("");
    } else if (slot >= 0) {
        const uint8_t* tile = cache_tile(c, slot, (int)h);
        const uint8_t* exps = tile + 2 * code_bytes(FMT, c.nb);
        const int t = (int)(slot & (kTile - 1));
        if (!value) {
            const float sc = ckpt_scale(exps[k_exp_at(c.nb, t, b)]);
            const uint8_t* at = tile + k_code_at(FMT, c.nb, t, b, g);
            uint32_t w[2];
            w[0] = *reinterpret_cast<const uint32_t*>(at);
            if constexpr (!four_bits(FMT)) w[1] = *reinterpret_cast<const uint32_t*>(at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = cache_decode2<FMT>(four_bits(FMT) ? w[0] >> (8 * i) & 0xFFu : w[i >> 1] >> (16 * (i & 1)) & 0xFFFFu, sc);
                y[2 * i] = v.x;
                y[2 * i + 1] = v.y;
            }
        } else {
            const float sc = ckpt_scale(exps[kTile * k_exp_bytes(c.nb) + v_exp_at(c.nb, t, b)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* at = tile + code_bytes(FMT, c.nb) + v_code_at(FMT, c.nb, t, b, 4 * g + i);
                const float2 v = cache_decode2<FMT>(four_bits(FMT) ? (uint32_t)*at : (uint32_t)*reinterpret_cast<const uint16_t*>(at), sc);
                y[i] = v.x;
                y[4 + i] = v.y;
            }
        }
    }
    Y* out = (value ? V : K) + (int64_t)row * c.d;
    if (!value) {
        store8(out + 8 * lane, y, c.d - 8 * lane);
        return;
    }
    // features 4 g + 0..3 of the block's two halves
    const int n = 32 * b + 4 * g;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        Y* at = out + n + 16 * half;
        const int left = c.d - n - 16 * half;
        f32x4 v = half ? f32x4{y[4], y[5], y[6], y[7]} : f32x4{y[0], y[1], y[2], y[3]};
        if constexpr (sizeof(Y) == 4) {
            if (left >= 4) *reinterpret_cast<f32x4u*>(at) = v;
            else
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < left) at[i] = v[i];
        } else {
            if (left >= 4) *reinterpret_cast<u16x4u*>(at) = u16x4u{bf16_bits(v[0]), bf16_bits(v[1]), bf16_bits(v[2]), bf16_bits(v[3])};
            else
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < left) at[i] = bf16_bits(v[i]);
        }
    }
}

// launch(the first workgroup, how many) for every piece of `groups` workgroups
template <typename F>
void in_pieces(uint32_t groups, F launch)
{
    for (uint32_t first = 0; first < groups;) {
        const uint32_t n = groups - first < kLaunchGroups ? groups - first : kLaunchGroups;
        launch(first, n);
        first += n;
    }
}

template <typename F>
void with_lanes(int lanes, F f)
{
    switch (lanes) {
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 8: f(std::integral_constant<int, 8>{}); break;
    case 16: f(std::integral_constant<int, 16>{}); break;
    case 32: f(std::integral_constant<int, 32>{}); break;
    default: f(std::integral_constant<int, 64>{}); break;
    }
}

}  // namespace

snack_status check_cache(const snack_cache* c, bool bare)
{
    if (!c || c->pages < 1 || c->heads < 1 || c->head_dim < 1 || c->head_dim > kMaxHeadDim || c->page_tokens < kTile ||
        c->page_tokens % kTile || !cache_format(c->fmt))
        return SNACK_ERR_INVALID_ARG;
    if (!bare && (!c->data || misaligned(c->data, 16))) return SNACK_ERR_INVALID_ARG;
    // tiles are numbered in 31 bits, and bytes stay within 63: tiles < 2^31, heads < 2^13, bytes of a tile < 2^15
    // (a quotient: the product of pages and tokens may pass 63 bits)
    if (c->pages > ((1ll << 36) - 1) / c->page_tokens || c->heads >= (1 << 13) ||
        (int64_t)c->heads * c->page_tokens >= (1ll << 31))
        return SNACK_ERR_UNSUPPORTED;
    return SNACK_OK;
}

void make_cache_view(const snack_cache* c, CacheView* v)
{
    v->data = c->data;
    v->slots = c->pages * c->page_tokens;
    v->page_tiles = c->page_tokens / kTile;
    v->heads = c->heads;
    v->d = c->head_dim;
    v->nb = cache_blocks(c->head_dim);
    v->record = tile_bytes(c->fmt, v->nb);
    v->by_page = fast_div((uint32_t)v->page_tiles);
    v->page_bytes = (int64_t)c->heads * v->page_tiles * v->record;
}

snack_status qk_pass(const QkPass& a, const CacheView* cache, int cache_fmt, int x_fmt, int y_fmt, int kclass,
                     hipStream_t s)
{
    ProfScope prof(kclass, s);
    QkPass b = a;
    b.inv_d = 1.0 / a.d;
    CacheView c{};
    if (cache) c = *cache;
    // heads of whole blocks, half of each turning with the other: the key path of whole pairs
    b.key_pairs = a.ro.table && a.ro.layout == SNACK_ROPE_HALF && a.ro.r % kCkptBlock == 0 && 2 * a.ro.r == a.d &&
                  cache_blocks(a.d) * kCkptBlock == a.d;
    const int hl = head_lanes(a.d), pl = pair_lanes(a.d, a.ro.r), lanes = hl > pl ? hl : pl;
    const uint32_t per = kThreads / lanes;
    const uint32_t gq = (a.q.rows + per - 1) / per, gk = (a.k.rows + per - 1) / per, gv = (a.v.rows + per - 1) / per;
    with_lanes(lanes, [&](auto n) {
        constexpr int LPR = decltype(n)::value;
        auto pick = [&](auto even) {
            constexpr bool EVEN = decltype(even)::value;
            if (x_fmt == SNACK_F32)
                return y_fmt == SNACK_F32 ? qk_pass_kernel<LPR, EVEN, float, float> : qk_pass_kernel<LPR, EVEN, float, uint16_t>;
            return y_fmt == SNACK_F32 ? qk_pass_kernel<LPR, EVEN, uint16_t, float> : qk_pass_kernel<LPR, EVEN, uint16_t, uint16_t>;
        };
        const auto k = even_lanes(a.d, a.ro.r) ? pick(std::true_type{}) : pick(std::false_type{});
        in_pieces(gq + gk + gv, [&](uint32_t first, uint32_t n) {
            hipLaunchKernelGGL(k, dim3(n), dim3(kThreads), 0, s, b, c, cache_fmt, gq, gk, first);
        });
    });
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

}  // namespace snack

using namespace snack;

extern "C" snack_status snack_cache_bytes(const snack_cache* cache, int64_t* bytes)
{
    if (!bytes) return SNACK_ERR_INVALID_ARG;
    SNACK_CHECK(check_cache(cache, true));
    CacheView c;
    make_cache_view(cache, &c);
    *bytes = cache->pages * c.page_bytes;
    return SNACK_OK;
}

extern "C" snack_status snack_cache_slots(const snack_cache* cache, const int32_t* table, int32_t width,
                                          const int32_t* lens, const int32_t* starts, int32_t sequences,
                                          int64_t tokens, int32_t* pos, int64_t* slot, snack_stream stream)
{
    SNACK_CHECK(check_cache(cache, true));
    if (width < 1 || sequences < 0 || tokens < 0) return SNACK_ERR_INVALID_ARG;
    if (tokens >= (1ll << 31)) return SNACK_ERR_UNSUPPORTED;
    if (tokens == 0) return SNACK_OK;
    if (!pos || !slot || misaligned(pos, 4) || misaligned(slot, 8)) return SNACK_ERR_INVALID_ARG;
    if (sequences && (!table || !lens || misaligned(table, 4) || misaligned(lens, 4) || misaligned(starts, 4)))
        return SNACK_ERR_INVALID_ARG;
    if (!starts && (sequences < 1 || tokens % sequences)) return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_CACHE, s);
    hipLaunchKernelGGL(slots_kernel, dim3((unsigned)((tokens + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, table,
                       width, lens, starts, sequences, (int32_t)(starts ? 1 : tokens / sequences), (int32_t)tokens,
                       cache->page_tokens, cache->pages, pos, slot);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

extern "C" snack_status snack_cache_write_rope(const snack_cache* cache, const void* Q, int64_t q_row, int64_t q_head,
                                               int32_t q_heads, const void* K, int64_t k_row, int64_t k_head,
                                               const void* V, int64_t v_row, int64_t v_head, int32_t x_fmt,
                                               int64_t tokens, const int32_t* pos, const int64_t* slot,
                                               const snack_rope* rope, const float* q_gain, const float* k_gain,
                                               float eps, void* Yq, int32_t y_fmt, snack_stream stream)
{
    SNACK_CHECK(check_cache(cache, false));
    QkPass a{};
    SNACK_CHECK(make_heads(Q, q_row, q_head, q_heads, tokens, cache->head_dim, x_fmt, &a.q));
    SNACK_CHECK(make_heads(K, k_row, k_head, cache->heads, tokens, cache->head_dim, x_fmt, &a.k));
    SNACK_CHECK(make_heads(V, v_row, v_head, cache->heads, tokens, cache->head_dim, x_fmt, &a.v));
    SNACK_CHECK(make_rotation(rope, cache->head_dim, pos, tokens, &a.ro));
    if (!float_format(y_fmt) || !(eps >= 0) || eps > 3.0e38f) return SNACK_ERR_INVALID_ARG;
    if (tokens == 0) return SNACK_OK;
    if (!K || !V || !slot || misaligned(slot, 8) || misaligned(q_gain, 4) || misaligned(k_gain, 4) ||
        (a.q.rows && (!Q || !Yq || misaligned(Yq, y_fmt == SNACK_F32 ? 4 : 2))))
        return SNACK_ERR_INVALID_ARG;
    a.d = cache->head_dim;
    a.pos = pos;
    a.slot = slot;
    a.q_gain = q_gain;
    a.k_gain = k_gain;
    a.eps = (double)eps;
    a.yq = Yq;
    CacheView c;
    make_cache_view(cache, &c);
    return qk_pass(a, &c, cache->fmt, x_fmt, y_fmt, KC_CACHE, reinterpret_cast<hipStream_t>(stream));
}

extern "C" snack_status snack_cache_write(const snack_cache* cache, const void* K, int64_t k_row, int64_t k_head,
                                          const void* V, int64_t v_row, int64_t v_head, int32_t x_fmt, int64_t tokens,
                                          const int64_t* slot, snack_stream stream)
{
    return snack_cache_write_rope(cache, nullptr, 0, 0, 0, K, k_row, k_head, V, v_row, v_head, x_fmt, tokens, nullptr,
                                  slot, nullptr, nullptr, nullptr, 0.0f, nullptr, SNACK_F32, stream);
}

extern "C" snack_status snack_cache_read(const snack_cache* cache, const int64_t* slot, int64_t tokens, void* K,
                                         void* V, int32_t y_fmt, snack_stream stream)
{
    SNACK_CHECK(check_cache(cache, false));
    Heads h;
    SNACK_CHECK(make_heads(nullptr, 0, 0, cache->heads, tokens, cache->head_dim, y_fmt, &h));
    if (tokens == 0) return SNACK_OK;
    const uintptr_t ya = y_fmt == SNACK_F32 ? 4 : 2;
    if (!slot || misaligned(slot, 8) || (!K && !V) || misaligned(K, ya) || misaligned(V, ya)) return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_CACHE, s);
    CacheView c;
    make_cache_view(cache, &c);
    const uint32_t per = kThreads / head_lanes(c.d), groups = (h.rows + per - 1) / per;
    const uint32_t gk = K ? groups : 0, gv = V ? groups : 0;
    with_lanes(head_lanes(c.d), [&](auto lanes) {
        constexpr int LPR = decltype(lanes)::value;
        auto launch = [&](auto fmt) {
            constexpr int FMT = decltype(fmt)::value;
            in_pieces(gk + gv, [&](uint32_t first, uint32_t n) {
                if (y_fmt == SNACK_F32)
                    hipLaunchKernelGGL((read_kernel<LPR, FMT, float>), dim3(n), dim3(kThreads), 0, s, c, slot, h.heads,
                                       h.rows, gk, first, (float*)K, (float*)V);
                else
                    hipLaunchKernelGGL((read_kernel<LPR, FMT, uint16_t>), dim3(n), dim3(kThreads), 0, s, c, slot, h.heads,
                                       h.rows, gk, first, (uint16_t*)K, (uint16_t*)V);
            });
        };
        if (cache->fmt == SNACK_INT8) launch(std::integral_constant<int, SNACK_INT8>{});
        else if (cache->fmt == SNACK_E4M3) launch(std::integral_constant<int, SNACK_E4M3>{});
        else launch(std::integral_constant<int, SNACK_E2M1>{});
    });
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}
