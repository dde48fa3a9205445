// attend.hip -- the attention's entry points: checks, workspace, launches.
#include "attend.h"

#include <math.h>

namespace snack {
namespace {

// what the launches need to know of a call before its lengths, which only the device knows
struct Plan {
    int kind;
    unsigned groups;
    int64_t units;    // at most
    int most;         // workgroups at most, and entries of the pieces' list
    int64_t part;     // floats of the partial results
    int64_t bytes;
};

// By the queries of a cache head that a sequence has on average.  Measured (us, both launches, int8, 32 query and 8
// cache heads of 128, 8192 tokens; blocks of 16 : 64 : 256 queries; bf16, fp32 queries): 4 sequences of 24 queries a
// head 39 : 38 : 59, 41 : 44 : 85; one of 96 30 : 28 : 35, 32 : 32 : 47; of 192 46 : 36 : 37, 49 : 41 : 52; of 384
// - : 53 : 51, - : 62 : 77; of 2048 - : 185 : 133, - : 230 : 214.  (fp32 queries would have blocks of 64 up to some 500.)
// Blocks of 256 of heads past 128 features would not fit the registers.  What is kept does not fit everywhere either:
// fp32 heads past 96 features in blocks of 256 spill 160 bytes a lane, heads past 160 in blocks of 64 up to 660 (four
// prompts of 2048 tokens, 8 heads, int8: of 128 features fp32 165 us, bf16 113; of 256 714 and 234).
int attend_kind(int nb, int64_t queries)
{
    if (queries <= kQueries) return kFew;
    return queries <= 128 || nb > 4 ? kMany64 : kMany256;
}

Plan make_plan(const CacheView& c, int32_t group, int64_t tokens, int32_t sequences, int64_t width)
{
    Plan p;
    p.kind = attend_kind(c.nb, sequences ? tokens * group / sequences : 0);
    const int rows = attend_rows(p.kind);
    // one workgroup of the largest kind a compute unit, two of the others
    const int most = p.kind == kMany256 ? kAttendGroups / 2 : kAttendGroups;
    // blocks of queries of every sequence and head at most, and their work (both factors below 2^31)
    p.units = c.heads * (tokens * group / rows + sequences);
    const int cost = p.kind == kFew ? kFewCost : kManyCost;
    const int64_t work = p.units * (width * c.page_tiles + 1 + cost);
    int64_t groups = (work + kMinRun - 1) / kMinRun;
    if (groups > most) groups = most;
    if (groups < 1) groups = 1;
    p.groups = (unsigned)groups;
    p.part = (int64_t)most * 2 * (rows / 16) * part_floats(c.nb);
    p.most = most;
    p.bytes = p.part * 4 + (2 * most + 1) * (int64_t)sizeof(int4);
    return p;
}

template <int QT, int ROWS>
void join(const AttendArgs& a, const Plan& p, hipStream_t s)
{
    const unsigned entries = a.by_unit ? (unsigned)p.units : p.groups;
    // Many pieces of each.  Measured (us, both launches; never : here : from two pieces on : always): one token over 131072
    // tokens 59 : 34 : 34 : 34, eight over 16384 39 : 39 : 36 : 36, 512 queries over 8192 135 : 135 : 149 : 149, four
    // prompts of 1024 56 : 56 : 56 : 81; from 32 pieces on 5 queries over 7 x 2000 22 against 17.
    if (p.units * 8 <= p.groups)
        hipLaunchKernelGGL((attend_join_kernel<QT, ROWS, true>), dim3(entries, ROWS / 16, 2 * a.c.nb), dim3(kAttendThreads), 0, s, a);
    else
        hipLaunchKernelGGL((attend_join_kernel<QT, ROWS, false>), dim3(entries, ROWS / 16), dim3(kAttendThreads), 0, s, a);
}
template <int QT>
void join(const AttendArgs& a, const Plan& p, hipStream_t s)
{
    switch (p.kind) {
    case kFew: join<QT, attend_rows(kFew)>(a, p, s); break;
    case kMany64: join<QT, attend_rows(kMany64)>(a, p, s); break;
    default: join<QT, attend_rows(kMany256)>(a, p, s); break;
    }
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
    const float scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (q_heads < 1 || q_heads % cache->heads || width < 1 || sequences < 0 || !(scale > 0) || !isfinite(scale_log2))
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
    a.most_blocks = (int32_t)(plan.units / cache->heads);
    a.hq = q_heads;
    a.by_group = fast_div((uint32_t)group);
    a.scale_log2 = scale_log2;
    a.causal = causal ? 1 : 0;
    a.part = (float*)work;
    a.meta = (int4*)(a.part + plan.part);
    a.by_unit = plan.units <= plan.most;
    a.meta_last = 2 * plan.most;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_ATTEND, s);
    if (cache->fmt == SNACK_INT8) SNACK_CHECK(launch_attend<SNACK_INT8>(a, q_fmt, plan.kind, plan.groups, s));
    else if (cache->fmt == SNACK_E4M3) SNACK_CHECK(launch_attend<SNACK_E4M3>(a, q_fmt, plan.kind, plan.groups, s));
    else SNACK_CHECK(launch_attend<SNACK_E2M1>(a, q_fmt, plan.kind, plan.groups, s));
    if (q_fmt == SNACK_F32) join<SNACK_F32>(a, plan, s);
    else join<SNACK_BF16>(a, plan, s);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}
