// rope.hip -- the table of the rotary positions, and the gradient of the norms and
// the rotation of queries and keys (the forward pass is cache.hip's: the same
// kernel also writes the cache).
//
//   y = x rstd gain for each head, rstd = 1 / sqrt(mean(x^2) + eps), then turned
//   dy = the gradient turned back, xh = x rstd, w = dy gain
//   dx = rstd (w - xh mean(w xh)),   dgain = sum over tokens and heads of dy xh
//
// One pass over x, the gradient and dx, which bounds it.  A head lies on a group of
// lanes, eight features each, so its two sums are a few DPP steps.  A workgroup
// takes a run of heads and adds up their terms of dgain in registers, in order; the
// partial rows of the workgroups are added up by a second launch in a fixed tree.
#include "rope.h"

#include <math.h>

namespace snack {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 1280;    // workgroups (and partial rows) of a gradient at most: five a compute unit, all at once
                                    // (2048: 71 against 62 us at 9001 tokens of 24 heads of 80)
constexpr int kSumThreads = 1024, kSumCols = 8;

__global__ void __launch_bounds__(kThreads) table_kernel(float* __restrict__ T, uint32_t total, FastDiv by_r,
                                                         double log2_base, double factor, double trained, double low,
                                                         double high, double amplitude)
{
    const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int r = (int)by_r.d;
    const uint32_t p = fast_quot(by_r, id), i = id - p * by_r.d;
    double f = exp2(-log2_base * (double)i / (double)r);
    double w = 0.0;
    if (trained > 0.0) w = fmin(fmax((trained * f * 0.15915494309189535 - low) / (high - low), 0.0), 1.0);
    f *= w + (1.0 - w) / factor;
    double s, c;
    sincos((double)p * f, &s, &c);
    float* row = T + (int64_t)p * (2 * r);
    row[i] = (float)(c * amplitude);
    row[r + i] = (float)(s * amplitude);
}

struct BwdPart {
    Heads x, g;          // x (p null: not read) and the gradient of y
    const float* gain;   // null: not normed
    void* dx;
    float* part;         // partial rows of dgain [groups][d], or null
    uint32_t groups;     // workgroups
    uint32_t run;        // heads (rows) of a workgroup
};

template <int LPR, bool EVEN, typename X, typename Y>
__global__ void __launch_bounds__(kThreads)
qk_bwd_kernel(BwdPart q, BwdPart k, int d, const int32_t* __restrict__ pos, Rotation ro, double eps, double inv_d)
{
    __shared__ float sums[kThreads * 8];
    const bool second = blockIdx.x >= q.groups;
    const BwdPart a = second ? k : q;
    const uint32_t group = second ? blockIdx.x - q.groups : blockIdx.x;
    constexpr int kRows = kThreads / LPR;
    const int lane = (int)threadIdx.x % LPR;
    const Spot8 at8 = find_spot8(lane, d, ro.r, ro.layout);
    const uint32_t first = group * a.run, last = min(a.x.rows, first + a.run);
    Eight gain{{0, 0, 0, 0}, {0, 0, 0, 0}}, dg = gain;
    if (a.gain) gain = take8<EVEN>(a.gain, at8, d);
    // whole wavefronts stay in the loop: the sums over lanes take every lane
    for (uint32_t at = first; at < last; at += kRows) {
        const uint32_t row = at + threadIdx.x / LPR;
        const bool live = row < last;
        const uint32_t rr = live ? row : last - 1;
        const uint32_t token = fast_quot(a.x.heads, rr), h = rr - token * a.x.heads.d;
        const int p = ro.table ? pos[token] : 0;
        Eight dy = take8<EVEN>((const Y*)a.g.p + (int64_t)token * a.g.row + (int64_t)h * a.g.head, at8, d);
        Eight x{{0, 0, 0, 0}, {0, 0, 0, 0}};
        if (a.gain) x = take8<EVEN>((const X*)a.x.p + (int64_t)token * a.x.row + (int64_t)h * a.x.head, at8, d);
        if (ro.table) {
            const Angles t = take_angles<EVEN>(ro, p, lane, at8.turned);
            const Eight g = dy;
            if (ro.layout == SNACK_ROPE_HALF || !at8.turned) {
                dy.a = g.a * t.c + g.b * t.s;
                dy.b = g.b * t.c - g.a * t.s;
            } else {
                dy.a = f32x4{g.a.x * t.c.x + g.a.y * t.s.x, g.a.y * t.c.x - g.a.x * t.s.x,
                             g.a.z * t.c.y + g.a.w * t.s.y, g.a.w * t.c.y - g.a.z * t.s.y};
                dy.b = f32x4{g.b.x * t.c.z + g.b.y * t.s.z, g.b.y * t.c.z - g.b.x * t.s.z,
                             g.b.z * t.c.w + g.b.w * t.s.w, g.b.w * t.c.w - g.b.z * t.s.w};
            }
            if (!at8.turned) {      // what is not turned keeps its own value, whatever its neighbours hold
                dy.a = g.a * t.c;
                dy.b = g.b * t.c;
            }
        }
        Eight dx = dy;
        if (a.gain) {
            const f32x4 wa = dy.a * gain.a, wb = dy.b * gain.b;
            // 64 bits: squares of any fp32 value
            double ss = 0.0, ws = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ss = fma((double)x.a[i], (double)x.a[i], ss);
                ss = fma((double)x.b[i], (double)x.b[i], ss);
                ws = fma((double)wa[i], (double)x.a[i], ws);
                ws = fma((double)wb[i], (double)x.b[i], ws);
            }
            const double v = fma(lanes_sum<LPR>(ss), inv_d, eps);
            const double r = v < __builtin_inf() ? rsqrt64(v) : v == v ? 0.0 : v;     // as the forward pass
            // Rows about the smallest normal numbers, without eps: 1 / rms is no fp32 number.  They are taken 2^64 times as
            // large, and their dx 2^64 times what that gives, both exact.
            const bool tiny = r >= 0x1p126, some = __ballot(tiny) != 0;
            const float up = tiny ? 0x1p64f : 1.0f;
            const double rs = tiny ? r * 0x1p-64 : r;
            if (some) {
                x.a *= up;
                x.b *= up;
            }
            const float rstd = (float)rs;
            const float m = (float)(lanes_sum<LPR>(ws) * inv_d * r * rs);
            if (live) {
                dg.a += dy.a * (x.a * rstd);
                dg.b += dy.b * (x.b * rstd);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dx.a[i] = rstd * fmaf(-x.a[i], m, wa[i]);
                dx.b[i] = rstd * fmaf(-x.b[i], m, wb[i]);
            }
            if (some) {
                dx.a *= up;
                dx.b *= up;
            }
        }
        if (live) {
            X* to = (X*)a.dx + (int64_t)row * d;
            put4(to + at8.a, dx.a, at8.na);
            put4(to + at8.b, dx.b, at8.nb);
        }
    }
    if (!a.part) return;
    // the threads of a feature: kRows of them, in order
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sums[i * kThreads + (int)threadIdx.x] = dg.a[i];
        sums[(4 + i) * kThreads + (int)threadIdx.x] = dg.b[i];
    }
    __syncthreads();
    for (int e = (int)threadIdx.x; e < 8 * LPR; e += kThreads) {
        const Spot8 to = find_spot8(e % LPR, d, ro.r, ro.layout);
        const int i = e / LPR;
        if ((i & 3) >= (i < 4 ? to.na : to.nb)) continue;
        float s = 0.0f;
        for (int j = 0; j < kRows; ++j) s += sums[i * kThreads + j * LPR + e % LPR];
        a.part[(int64_t)group * d + (i < 4 ? to.a : to.b) + (i & 3)] = s;
    }
}

// dgain[f] = sum over the partial rows, in 64 bits; a workgroup 8 features, its threads 128 runs of rows each
__global__ void __launch_bounds__(kSumThreads)
gain_sum_kernel(const float* __restrict__ pq, uint32_t nq, float* __restrict__ gq, const float* __restrict__ pk,
                uint32_t nk, float* __restrict__ gk, int d)
{
    __shared__ double sums[kSumThreads / kSumCols][kSumCols + 1];
    const bool second = blockIdx.y != 0;
    const float* p = second ? pk : pq;
    const uint32_t n = second ? nk : nq;
    float* out = second ? gk : gq;
    if (!out) return;
    constexpr uint32_t kRuns = kSumThreads / kSumCols;
    const int c = (int)threadIdx.x % kSumCols, f = (int)blockIdx.x * kSumCols + c;
    const uint32_t r = threadIdx.x / kSumCols;
    double s = 0.0;
    if (f < d)
#pragma unroll 8
        for (uint32_t i = r; i < n; i += kRuns) s += p[(int64_t)i * d + f];
    sums[r][c] = s;
    __syncthreads();
    for (uint32_t half = kRuns / 2; half; half >>= 1) {
        if (r < half) sums[r][c] += sums[r + half][c];
        __syncthreads();
    }
    if (r == 0 && f < d) out[f] = (float)sums[0][c];
}

// workgroups of `rows` heads and the heads of each
void bwd_split(uint32_t rows, int lanes, uint32_t most, uint32_t* groups, uint32_t* run)
{
    const uint32_t per = kThreads / lanes;
    const uint32_t units = (rows + per - 1) / per;     // rows a workgroup takes at once
    const uint32_t turns = units ? (units + most - 1) / most : 0;
    *run = turns * per;
    *groups = turns ? (units + turns - 1) / turns : 0;
}
// of queries and keys: the workgroups shared out by their heads
void bwd_splits(uint32_t rq, uint32_t rk, int lanes, uint32_t* gq, uint32_t* runq, uint32_t* gk, uint32_t* runk)
{
    const uint64_t all = (uint64_t)rq + rk;
    const uint32_t mq = all ? (uint32_t)((uint64_t)kMaxGroups * rq / all) : 0;
    bwd_split(rq, lanes, mq < 1 ? 1 : mq, gq, runq);
    bwd_split(rk, lanes, kMaxGroups - mq < 1 ? 1 : kMaxGroups - mq, gk, runk);
}

}  // namespace

snack_status make_heads(const void* p, int64_t row, int64_t head, int32_t heads, int64_t tokens, int32_t d, int32_t fmt,
                        Heads* out)
{
    if (heads < 0 || tokens < 0 || d < 1 || d > 256 || !float_format(fmt)) return SNACK_ERR_INVALID_ARG;
    if (tokens >= (1ll << 31) || tokens * heads >= (1ll << 31)) return SNACK_ERR_UNSUPPORTED;
    out->p = p;
    out->row = row;
    out->head = head;
    out->heads = fast_div((uint32_t)(heads < 1 ? 1 : heads));
    out->rows = (uint32_t)(tokens * heads);
    if (out->rows && misaligned(p, fmt == SNACK_F32 ? 4 : 2)) return SNACK_ERR_INVALID_ARG;
    return SNACK_OK;
}

snack_status make_rotation(const snack_rope* rope, int32_t d, const int32_t* pos, int64_t tokens, Rotation* out)
{
    *out = Rotation{nullptr, 0, 0, 0};
    if (!rope) return SNACK_OK;
    if (!rope->table || rope->positions < 1 || rope->rot < 2 || rope->rot % 2 || rope->rot > d || (tokens && !pos))
        return SNACK_ERR_INVALID_ARG;
    if (rope->layout != SNACK_ROPE_HALF && rope->layout != SNACK_ROPE_PAIRS) return SNACK_ERR_INVALID_ARG;
    if (misaligned(rope->table, 4) || misaligned(pos, 4)) return SNACK_ERR_INVALID_ARG;
    *out = Rotation{rope->table, (uint32_t)rope->positions, rope->rot / 2, rope->layout};
    return SNACK_OK;
}

}  // namespace snack

using namespace snack;

extern "C" snack_status snack_rope_table(int32_t positions, int32_t rot, double base, double factor, double trained,
                                         double low, double high, double amplitude, float* table, snack_stream stream)
{
    if (positions < 1 || rot < 2 || rot % 2 || rot > 256 || !table || misaligned(table, 4)) return SNACK_ERR_INVALID_ARG;
    if (!(base > 0) || !(factor > 0) || !(trained >= 0) || !(low < high) || !isfinite(base) || !isfinite(factor) ||
        !isfinite(trained) || !isfinite(low) || !isfinite(high) || !isfinite(amplitude))
        return SNACK_ERR_INVALID_ARG;
    const int64_t total = (int64_t)positions * (rot / 2);
    if (total >= (1ll << 31)) return SNACK_ERR_UNSUPPORTED;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_ROPE, s);
    hipLaunchKernelGGL(table_kernel, dim3((unsigned)((total + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, table,
                       (uint32_t)total, fast_div((uint32_t)(rot / 2)), log2(base), factor, trained, low, high,
                       amplitude);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

extern "C" snack_status snack_qk_rope_fwd(const void* Q, int64_t q_row, int64_t q_head, int32_t q_heads, const void* K,
                                          int64_t k_row, int64_t k_head, int32_t k_heads, int32_t x_fmt,
                                          int64_t tokens, int32_t head_dim, const int32_t* pos, const snack_rope* rope,
                                          const float* q_gain, const float* k_gain, float eps, void* Yq, void* Yk,
                                          int32_t y_fmt, snack_stream stream)
{
    QkPass a{};
    SNACK_CHECK(make_heads(Q, q_row, q_head, q_heads, tokens, head_dim, x_fmt, &a.q));
    SNACK_CHECK(make_heads(K, k_row, k_head, k_heads, tokens, head_dim, x_fmt, &a.k));
    SNACK_CHECK(make_rotation(rope, head_dim, pos, tokens, &a.ro));
    if (!float_format(y_fmt) || !(eps >= 0) || !isfinite(eps)) return SNACK_ERR_INVALID_ARG;
    if (tokens == 0) return SNACK_OK;
    const uintptr_t ya = y_fmt == SNACK_F32 ? 4 : 2;
    if ((a.q.rows && (!Q || !Yq || misaligned(Yq, ya))) || (a.k.rows && (!K || !Yk || misaligned(Yk, ya))) ||
        misaligned(q_gain, 4) || misaligned(k_gain, 4) || a.q.rows + (uint64_t)a.k.rows == 0)
        return SNACK_ERR_INVALID_ARG;
    a.d = head_dim;
    a.pos = pos;
    a.q_gain = q_gain;
    a.k_gain = k_gain;
    a.eps = (double)eps;
    a.yq = Yq;
    a.yk = Yk;
    return qk_pass(a, nullptr, 0, x_fmt, y_fmt, KC_ROPE, reinterpret_cast<hipStream_t>(stream));
}

extern "C" snack_status snack_qk_rope_bwd_work(int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                                               int64_t* bytes)
{
    Heads q, k;
    if (!bytes) return SNACK_ERR_INVALID_ARG;
    SNACK_CHECK(make_heads(nullptr, 0, 0, q_heads, tokens, head_dim, SNACK_F32, &q));
    SNACK_CHECK(make_heads(nullptr, 0, 0, k_heads, tokens, head_dim, SNACK_F32, &k));
    // the lanes of a head, and with them the workgroups, depend on the rotation: no more than the workgroups' limit
    // (each side's share rounded up) or a workgroup for the fewest heads that one takes
    uint64_t groups = kMaxGroups + 2;
    const uint64_t fewest = ((uint64_t)q.rows + k.rows + 3) / 4 + 2;
    if (fewest < groups) groups = fewest;
    *bytes = (int64_t)groups * head_dim * 4;
    return SNACK_OK;
}

extern "C" snack_status snack_qk_rope_bwd(const void* Q, int64_t q_row, int64_t q_head, int32_t q_heads, const void* K,
                                          int64_t k_row, int64_t k_head, int32_t k_heads, int32_t x_fmt,
                                          int64_t tokens, int32_t head_dim, const int32_t* pos, const snack_rope* rope,
                                          const float* q_gain, const float* k_gain, float eps, const void* dYq,
                                          int64_t dq_row, int64_t dq_head, const void* dYk, int64_t dk_row,
                                          int64_t dk_head, int32_t y_fmt, void* dXq, void* dXk, float* dq_gain,
                                          float* dk_gain, void* work, int64_t work_bytes, snack_stream stream)
{
    BwdPart q{}, k{};
    Rotation ro;
    SNACK_CHECK(make_heads(q_gain ? Q : nullptr, q_row, q_head, q_heads, tokens, head_dim, x_fmt, &q.x));
    SNACK_CHECK(make_heads(k_gain ? K : nullptr, k_row, k_head, k_heads, tokens, head_dim, x_fmt, &k.x));
    SNACK_CHECK(make_heads(dYq, dq_row, dq_head, q_heads, tokens, head_dim, y_fmt, &q.g));
    SNACK_CHECK(make_heads(dYk, dk_row, dk_head, k_heads, tokens, head_dim, y_fmt, &k.g));
    SNACK_CHECK(make_rotation(rope, head_dim, pos, tokens, &ro));
    if (!(eps >= 0) || !isfinite(eps) || (dq_gain && !q_gain) || (dk_gain && !k_gain)) return SNACK_ERR_INVALID_ARG;
    const uintptr_t xa = x_fmt == SNACK_F32 ? 4 : 2;
    if ((q.x.rows && (!dYq || !dXq || misaligned(dXq, xa) || (q_gain && !Q))) ||
        (k.x.rows && (!dYk || !dXk || misaligned(dXk, xa) || (k_gain && !K))) || misaligned(q_gain, 4) ||
        misaligned(k_gain, 4) || misaligned(dq_gain, 4) || misaligned(dk_gain, 4) || q_heads + (int64_t)k_heads == 0)
        return SNACK_ERR_INVALID_ARG;
    const int lanes = pair_lanes(head_dim, ro.r);
    bwd_splits(q.x.rows, k.x.rows, lanes, &q.groups, &q.run, &k.groups, &k.run);
    if (dq_gain || dk_gain) {
        const int64_t need = ((int64_t)q.groups + k.groups) * head_dim * 4;
        if (need && (!work || misaligned(work, 4))) return SNACK_ERR_INVALID_ARG;
        if (work_bytes < need) return SNACK_ERR_WORKSPACE;
        if (dq_gain) q.part = (float*)work;
        if (dk_gain) k.part = (float*)work + (int64_t)q.groups * head_dim;
    }
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_ROPE, s);
    q.gain = q_gain;
    k.gain = k_gain;
    q.dx = dXq;
    k.dx = dXk;
    const unsigned groups = q.groups + k.groups;
    if (groups) {
        auto launch = [&](auto lanes, auto x, auto y) {
            constexpr int LPR = decltype(lanes)::value;
            const auto kernel = even_lanes(head_dim, ro.r) ? qk_bwd_kernel<LPR, true, decltype(x), decltype(y)>
                                                           : qk_bwd_kernel<LPR, false, decltype(x), decltype(y)>;
            hipLaunchKernelGGL(kernel, dim3(groups), dim3(kThreads), 0, s, q, k, head_dim, pos, ro, (double)eps,
                               1.0 / head_dim);
        };
        auto types = [&](auto lanes) {
            if (x_fmt == SNACK_F32) {
                if (y_fmt == SNACK_F32) launch(lanes, float{}, float{});
                else launch(lanes, float{}, uint16_t{});
            } else {
                if (y_fmt == SNACK_F32) launch(lanes, uint16_t{}, float{});
                else launch(lanes, uint16_t{}, uint16_t{});
            }
        };
        switch (lanes) {
        case 4: types(std::integral_constant<int, 4>{}); break;
        case 8: types(std::integral_constant<int, 8>{}); break;
        case 16: types(std::integral_constant<int, 16>{}); break;
        case 32: types(std::integral_constant<int, 32>{}); break;
        default: types(std::integral_constant<int, 64>{}); break;
        }
        SNACK_HIP(hipGetLastError());
    }
    if (dq_gain || dk_gain) {
        hipLaunchKernelGGL(gain_sum_kernel, dim3((unsigned)((head_dim + kSumCols - 1) / kSumCols), 2), dim3(kSumThreads), 0, s, q.part,
                           q.groups, dq_gain, k.part, k.groups, dk_gain, head_dim);
        SNACK_HIP(hipGetLastError());
    }
    return SNACK_OK;
}
