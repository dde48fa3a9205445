// cache.h -- the layout of the key/value cache and its block formats, on the device.
//
// Values are kept in blocks of 32 consecutive features of one token's head, as in
// the activation checkpoints: 32 codes and one exponent byte s, a code c standing
// for c 2^(s - 127); c is a signed integer (SNACK_INT8), an e4m3 number
// (SNACK_E4M3) or an e2m1 number (SNACK_E2M1, 4 bits).  A block that holds a NaN
// or an infinity has s = 255 and codes 0 and reads back as NaN.
//
// The codes lie in the order in which the attention's matrix instructions take
// them, so that a wavefront reads whole contiguous kilobytes straight into operand
// registers: no transposition and no LDS between memory and the instruction.  A
// tile is 32 tokens of one head, a page a whole number of tiles:
//   data[page][head][tile]: K codes | V codes | K exponents | V exponents
// The instruction (16x16x32, bf16) takes as its first operand 16 rows of 32 values;
// lane l holds row l % 16, values 8 (l / 16) + 0..7.
//   scores   S^T = K Q^T: rows are 16 tokens, values 32 features (one block).  Token
//            t of the tile is row 4 (t / 8) + t % 4 of half (t / 4) % 2; then the
//            lane that gets the scores of a query (its column) for rows 4 g + 0..3
//            of both halves has tokens 8 g + 0..7, which is what
//   output   O^T = V^T P^T takes as its second operand from that lane: rows are 16
//            features, values the 32 tokens of the tile.
// The scores never leave their lane between the two products.  A V byte pair (byte,
// for 4 bits) holds features d and d + 16 of one token, which share the scale that
// the conversion instruction applies to both.
#pragma once

#include "ckpt.h"

namespace snack {

constexpr int kTile = 32;          // tokens of a tile
constexpr int kMaxHeadDim = 256;   // largest features of a head

__host__ __device__ constexpr bool four_bits(int fmt) { return fmt == SNACK_E2M1; }
inline bool cache_format(int32_t fmt) { return fmt == SNACK_INT8 || fmt == SNACK_E4M3 || fmt == SNACK_E2M1; }
// bytes of a token's K exponents: blocks of a head rounded up to what one load takes
__host__ __device__ constexpr int k_exp_bytes(int nb) { return nb <= 1 ? 1 : nb <= 2 ? 2 : nb <= 4 ? 4 : 8; }
__host__ __device__ constexpr int code_bytes(int fmt, int nb) { return kTile * nb * (four_bits(fmt) ? 16 : 32); }
__host__ __device__ constexpr int tile_bytes(int fmt, int nb)
{
    return 2 * code_bytes(fmt, nb) + kTile * k_exp_bytes(nb) + kTile * nb;
}

// where the codes of token t's features 32 b + 8 g + 0..7 start among the K codes (8 bytes, or 4)
__host__ __device__ constexpr int k_code_at(int fmt, int nb, int t, int b, int g)
{
    const int half = (t >> 2) & 1, lane = 4 * (t >> 3) + (t & 3) + 16 * g;
    const int per = four_bits(fmt) ? 4 : 2, unit = four_bits(fmt) ? 4 : 8;   // blocks of a 16-byte chunk, bytes of each
    const int c = b / per, w = nb - per * c < per ? nb - per * c : per;
    return half * (kTile / 2) * nb * 4 * unit + c * 1024 + (lane * w + b % per) * unit;
}
// where the code of token t's feature 32 b + n lies among the V codes, n < 16 (the byte after it, or the
// high four bits, hold feature 32 b + n + 16)
__host__ __device__ constexpr int v_code_at(int fmt, int nb, int t, int b, int n)
{
    const int lane = n + 16 * (t >> 3);
    if (!four_bits(fmt)) return b * 1024 + lane * 16 + 2 * (t & 7);
    const int c = b / 2, w = nb - 2 * c < 2 ? 1 : 2;
    return c * 1024 + lane * 8 * w + 8 * (b & 1) + (t & 7);
}
// among the exponents: token t's block b
__host__ __device__ constexpr int k_exp_at(int nb, int t, int b)
{
    return (((t >> 2) & 1) * 16 + 4 * (t >> 3) + (t & 3)) * k_exp_bytes(nb) + b;
}
__host__ __device__ constexpr int v_exp_at(int nb, int t, int b) { return ((t >> 3) * nb + b) * 8 + (t & 7); }

// A cache as a kernel takes it.
struct CacheView {
    uint8_t* data;
    int64_t slots;         // tokens it has room for: pages * tokens of a page
    int32_t page_tiles;    // tiles of a page
    int32_t heads, d, nb;
    int32_t record;        // bytes of a tile
    FastDiv by_page;       // tiles -> pages
    int64_t page_bytes;
};

// the tile of slot `slot` (a token's place: page * tokens of a page + its offset) and head h
__device__ inline uint8_t* cache_tile(const CacheView& c, int64_t slot, int h)
{
    const uint32_t tile = (uint32_t)(slot / kTile), page = fast_quot(c.by_page, tile);
    return c.data + (int64_t)page * c.page_bytes + ((int64_t)h * c.page_tiles + (tile - page * c.page_tiles)) * c.record;
}

// the exponent byte of a block whose largest |x| has these bits
template <int FMT>
__device__ inline uint32_t cache_exponent(uint32_t amax)
{
    if constexpr (FMT != SNACK_E2M1) {
        return ckpt_exponent<FMT>(amax);
    } else {
        const int e = (int)(amax >> 23);                                // 6 = 1.5 * 2^2
        const int s = e - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        return e == 255 ? 255u : (uint32_t)(s < 1 ? 1 : s);
    }
}

// Two codes from two values, in the low bits of the result (16 of them, or 8), rounded once, nearest even.
// e2m1: the conversion takes the scale itself (its exponent bits alone).
template <int FMT>
__device__ inline uint32_t cache_encode2(float a, float b, uint32_t s)
{
    uint32_t w;
    if constexpr (FMT == SNACK_E2M1) {
        const float inv = ckpt_inverse(s);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a * inv, b * inv, 1.0f, 0) & 0xFFu;
    } else {
        w = ckpt_encode4<FMT>(f32x4{a, b, 0.0f, 0.0f}, s) & 0xFFFFu;
    }
    return s == 255u ? 0u : w;
}

// the values of two codes (the low 16 or 8 bits of w), times the block's scale
template <int FMT>
__device__ inline float2 cache_decode2(uint32_t w, float scale)
{
    if constexpr (FMT == SNACK_E2M1) {
        const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        return make_float2(v[0] * scale, v[1] * scale);
    } else {
        const f32x4 v = ckpt_codes4<FMT>(w);
        return make_float2(v.x * scale, v.y * scale);
    }
}

// blocks of a head as the kernels take them (the instances that there are; what is past the head's is zero)
__host__ __device__ constexpr int cache_blocks(int d)
{
    const int nb = (d + kCkptBlock - 1) / kCkptBlock;
    return nb == 5 ? 6 : nb == 7 ? 8 : nb;
}
void make_cache_view(const snack_cache* c, CacheView* v);
// whether a cache's description holds together (its data may be absent where `bare`)
snack_status check_cache(const snack_cache* c, bool bare);

}  // namespace snack
