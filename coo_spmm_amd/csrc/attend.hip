// attend.hip -- the attention's entry points: checks, workspace, launches.
#include "attend.h"

#include <math.h>

namespace snack {
namespace {

constexpr int kGroups = 512;   // workgroups at most: two a compute unit

// what the launches need to know of a call before its lengths, which only the device knows
struct Plan {
    int kind;
    unsigned groups;
    int64_t part;     // floats of the partial results
    int64_t bytes;
};

// by the queries of a cache head that a sequence has on average
int attend_kind(int nb, int64_t queries)
{
    if (queries <= kQueries) return kFew;
    return queries <= 64 || nb > 4 ? kMany64 : kMany128;
}

Plan make_plan(const CacheView& c, int32_t group, int64_t tokens, int32_t sequences, int64_t width)
{
    Plan p;
    p.kind = attend_kind(c.nb, sequences ? tokens * group / sequences : 0);
    const int rows = attend_rows(p.kind);
    // blocks of queries of every sequence and head at most, and their tiles (both below 2^31)
    const int64_t units = c.heads * (tokens * group / rows + sequences);
    const int64_t tiles = units * (width * c.page_tiles + 1);
    int64_t groups = (tiles + kMinRun - 1) / kMinRun;
    if (groups > kGroups) groups = kGroups;
    if (groups < 1) groups = 1;
    p.groups = (unsigned)groups;
    p.part = (int64_t)kGroups * 2 * (rows / 16) * part_floats(c.nb);
    p.bytes = p.part * 4 + kGroups * (int64_t)sizeof(int4);
    return p;
}

template <int QT>
auto join_kernel(int kind)
{
    return kind == kFew ? attend_join_kernel<QT, attend_rows(kFew)>
           : kind == kMany64 ? attend_join_kernel<QT, attend_rows(kMany64)> : attend_join_kernel<QT, attend_rows(kMany128)>;
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" snack_status snack_cache_attend_work(const snack_cache* cache, int32_t q_heads, int64_t tokens,
                                                int32_t sequences, int64_t* bytes)
{
    SNACK_CHECK(check_cache(cache, true));
    if (!bytes || q_heads < 1 || q_heads % cache->heads || tokens < 0 || sequences < 0) return SNACK_ERR_INVALID_ARG;
    if (tokens >= (1ll << 31) || tokens * q_heads >= (1ll << 31)) return SNACK_ERR_UNSUPPORTED;
    CacheView c;
    make_cache_view(cache, &c);
    *bytes = make_plan(c, q_heads / cache->heads, tokens, sequences, 1).bytes;
    return SNACK_OK;
}

extern "C" snack_status snack_cache_attend(const snack_cache* cache, const void* Q, int64_t q_row, int64_t q_head,
                                           int32_t q_heads, int32_t q_fmt, int64_t tokens, const int32_t* table,
                                           int32_t width, const int32_t* lens, const int32_t* starts,
                                           int32_t sequences, float scale, int32_t causal, void* out, void* work,
                                           int64_t work_bytes, snack_stream stream)
{
    SNACK_CHECK(check_cache(cache, false));
    if (q_heads < 1 || q_heads % cache->heads || width < 1 || sequences < 0 || !(scale > 0) || !isfinite(scale))
        return SNACK_ERR_INVALID_ARG;
    Heads q;
    SNACK_CHECK(make_heads(Q, q_row, q_head, q_heads, tokens, cache->head_dim, q_fmt, &q));
    // sequences x heads x blocks of queries are numbered in 31 bits; pages of a cache's table too
    if ((int64_t)sequences * cache->heads + q.rows >= (1ll << 31) || cache->pages >= (1ll << 31) ||
        (int64_t)width * (cache->page_tokens / kTile) >= (1ll << 31) - 1)
        return SNACK_ERR_UNSUPPORTED;
    if (tokens == 0 || (sequences == 0 && starts)) return SNACK_OK;
    if (!starts && (sequences < 1 || tokens % sequences)) return SNACK_ERR_INVALID_ARG;
    const uintptr_t qa = q_fmt == SNACK_F32 ? 4 : 2;
    if (!Q || !out || !table || !lens || misaligned(out, qa) || misaligned(table, 4) || misaligned(lens, 4) ||
        misaligned(starts, 4) || !work || misaligned(work, 16))
        return SNACK_ERR_INVALID_ARG;
    AttendArgs a{};
    make_cache_view(cache, &a.c);
    const int32_t group = q_heads / cache->heads;
    const Plan plan = make_plan(a.c, group, tokens, sequences, width);
    if (work_bytes < plan.bytes) return SNACK_ERR_WORKSPACE;
    a.q = Q;
    a.q_row = q_row;
    a.q_head = q_head;
    a.out = out;
    a.table = table;
    a.width = width;
    a.pages = (int32_t)cache->pages;
    a.lens = lens;
    a.starts = starts;
    a.sequences = sequences;
    a.per = starts ? 0 : (int32_t)(tokens / sequences);
    a.tokens = (int32_t)tokens;
    a.hq = q_heads;
    a.by_group = fast_div((uint32_t)group);
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.causal = causal ? 1 : 0;
    a.part = (float*)work;
    a.meta = (int4*)(a.part + plan.part);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_ATTEND, s);
    if (cache->fmt == SNACK_INT8) SNACK_CHECK(launch_attend<SNACK_INT8>(a, q_fmt, plan.kind, plan.groups, s));
    else if (cache->fmt == SNACK_E4M3) SNACK_CHECK(launch_attend<SNACK_E4M3>(a, q_fmt, plan.kind, plan.groups, s));
    else SNACK_CHECK(launch_attend<SNACK_E2M1>(a, q_fmt, plan.kind, plan.groups, s));
    const auto join = q_fmt == SNACK_F32 ? join_kernel<SNACK_F32>(plan.kind) : join_kernel<SNACK_BF16>(plan.kind);
    hipLaunchKernelGGL(join, dim3(plan.groups, 2 * a.c.nb, attend_rows(plan.kind) / 16), dim3(kAttendThreads), 0, s, a);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}
