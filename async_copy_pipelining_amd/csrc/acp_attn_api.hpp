// Entry points of attention over a paged cache.  Included by acp_entry.cpp
// after acp_heads_api.hpp, whose helpers it uses.
#include <limits>

#include "acp_attn.hpp"

namespace {

// Workgroups that the device has room for at a time: two a CU; one of 256 channels
// or of eight waves.
constexpr int64_t kAttendGroups = 512;
constexpr int64_t kAttendGroupsWide = 256;
// Fewer tiles than workgroups are dealt out evenly; others are a workgroup's each:
// shares begin inside tiles, so that neighbours no longer read the same keys at
// the same time ([2 x 4096, 16 heads, 64] as 848 tiles: 89 us, in shares 109).
// Keys of a share, at least ([4 tokens over up to 2000 positions, 32 / 8 heads,
// 128]: 20 us, of 512 24, of 128 18; one token over 32768: 38, 36 and 45).
constexpr int64_t kAttendLeast = 256;
// Sequences of at most so many positions are a workgroup's each, however few (4
// tokens over up to 1000 positions 18 us, dealt out 19; over 2000 36, dealt out 20).
constexpr int64_t kAttendAlone = 1024;
// Neighbouring heads in a workgroup, at most 2^k of them (32 tokens over up to
// 32768 positions 403 us; two heads 418, one 453).
constexpr int64_t kAttendSide = 2;
// Rows of a sequence from which on the form for many is taken.  The other has 16
// of a tile, and reads the keys for each: where all sequences have the same number
// its limit is one tile ([64 tokens over up to 8192 positions, 32 / 2 heads] 70 us,
// many rows 86; 48 / 2 heads 111, 88), and on average of sequences that differ less
// (16 of up to 8192 positions, 32 / 8 heads: 10 rows 82 us, 89; 15 rows 101, 90).
// 8-bit rows become 16 bits on their way to the form for many: three tiles
// (30 rows 89 us, 110).
constexpr int64_t kAttendPrompt = acp::kStepRows + 1, kAttendPromptRagged = 12, kAttendPrompt8 = 44;

struct AttendPlan {
  acp::AttendArgs A{};
  acp::JoinShape join{};
  int tile_rows = 0, padded = 0, cache = 0, dt = 0;
  int64_t workspace = 0, tokens = 0;
  int64_t stat_at = 0, joins_at = 0;
};

// Everything but addresses: shapes, the form, the split of the keys.
acp_status attend_plan(const acp::DescData& q, const CacheSide& k, const acp_sequences* b, AttendPlan* P) {
  acp::AttendArgs& A = P->A;
  const int64_t heads = heads_of(q), kv = k.d.shape[2], dim = dim_of(q);
  P->tokens = tokens_of(q);
  if (q.dtype == ACP_F32) return ret(ACP_ERR_UNSUPPORTED, "attention takes f16 or bf16");
  if (k.kind == acp::kCacheSame && k.d.dtype != q.dtype)
    return ret(ACP_ERR_INVALID, "the queries and the cache differ in dtype");
  if (k.d.shape[3] != dim) return ret(ACP_ERR_INVALID, "the queries and the cache differ in channels");
  if (dim < 8 || dim > 256 || dim % 8)
    return ret(ACP_ERR_UNSUPPORTED, "attention takes heads of 8 to 256 channels in multiples of 8");
  if (kv < 1 || heads % kv) return ret(ACP_ERR_INVALID, "the cache's heads must divide the queries'");
  const acp_status st = load_batch(b, k, &A.batch);
  if (st != ACP_OK) return st;
  if (heads >= kRowLimit || P->tokens >= kRowLimit || P->tokens * heads >= kRowLimit)
    return ret(ACP_ERR_UNSUPPORTED, "2^31 rows of queries");
  P->dt = row_dtype(q.dtype);
  P->cache = k.kind;
  P->padded = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  A.tokens = static_cast<uint32_t>(P->tokens);
  A.dim = static_cast<uint32_t>(dim);
  const int64_t group = std::max<int64_t>(1, heads / kv), sequences = b->sequences;
  A.group = div_by(static_cast<uint64_t>(group));
  if (P->tokens == 0 || heads == 0 || sequences == 0) return ACP_OK;
  // rows of a sequence: its tokens' query heads of one of the cache's
  const int64_t rows = b->starts ? P->tokens * group : sequences * group;
  const int64_t many = k.kind != acp::kCacheSame                   ? kAttendPrompt8
                       : b->starts && P->tokens > sequences ? kAttendPromptRagged
                                                            : kAttendPrompt;
  P->tile_rows = rows >= many * sequences ? 32 * acp::prompt_waves(P->padded) : acp::kStepRows;
  const int64_t M = P->tile_rows;
  const int64_t slots = b->starts ? P->tokens * group / M + sequences : sequences * ceil_div(group, M);
  if (slots >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 tiles of rows");
  A.slots = div_by(static_cast<uint64_t>(slots));
  // the longest that a sequence can be
  int64_t longest = std::min<int64_t>(int64_t(b->max_pages) * k.d.shape[1], (int64_t(1) << 31) - 1);
  if (b->max_length) longest = std::min<int64_t>(longest, b->max_length);
  const int64_t groups = P->padded == 256 || M == 256 ? kAttendGroupsWide : kAttendGroups;
  // sequences mostly fill fewer tiles than their slots
  const int64_t tiles = std::max<int64_t>(sequences, b->starts ? P->tokens * group / M : slots);
  // few rows: neighbouring heads, whose rows lie side by side, in the waves of a
  // workgroup, as long as all workgroups have work
  while (M == acp::kStepRows && A.side_log2 < kAttendSide && kv % (int64_t(2) << A.side_log2) == 0 &&
         (kv >> (A.side_log2 + 1)) * tiles * ceil_div(longest, kAttendLeast) >= groups)
    ++A.side_log2;
  const int64_t heads_each = kv >> A.side_log2;
  A.once = rows <= M * sequences;
  A.kv_heads = div_by(static_cast<uint64_t>(heads_each));
  int64_t grid = heads_each * slots;
  if (heads_each * tiles < groups && longest > kAttendAlone) {
    const int64_t most = std::max<int64_t>(1, groups / heads_each);
    A.shares = static_cast<uint32_t>(std::min(most, slots * ceil_div(longest + 1, kAttendLeast)));
    A.least = static_cast<uint32_t>(kAttendLeast);
    grid = heads_each * A.shares;
    const int64_t rows = grid * 2 * (M << A.side_log2);
    P->stat_at = rows * dim * 4;
    P->joins_at = P->stat_at + rows * 8;
    P->workspace = P->joins_at + heads_each * slots * 8;
    // the join: at most four partial results in a row for a lane, as long as lanes last
    const int64_t used = A.side_log2 || b->starts ? M << A.side_log2 : std::min(M, group);
    int lanes = 4, shares = 0;
    while ((int64_t(4) << lanes) < dim) ++lanes;
    while (lanes + shares < 8 && (int64_t(4) << shares) < ceil_div(A.shares, tiles) + 1) ++shares;
    P->join.lanes_log2 = lanes;
    P->join.shares_log2 = shares;
    const int64_t blocks = ceil_div(used, acp::kAttendThreads >> (lanes + shares));
    P->join.blocks = div_by(static_cast<uint64_t>(blocks));
    grid = std::max(grid, heads_each * slots * blocks);
  }
  const int64_t threads = M == acp::kStepRows ? acp::kAttendThreads : 64 * acp::prompt_waves(P->padded);
  if (grid * threads >= int64_t(1) << 32) return ret(ACP_ERR_UNSUPPORTED, "a launch of 2^32 lanes");
  return ACP_OK;
}

acp_status cache_attention_workspace(const acp_tile_desc* q, const acp_paged_cache* cache, const acp_sequences* b,
                                     int64_t* bytes) {
  acp::DescData qd;
  CacheSide k, v;
  AttendPlan P;
  if (!bytes) return ret(ACP_ERR_INVALID, "null argument");
  acp_status st = load_heads(q, "q", &qd);
  if (st == ACP_OK) st = load_cache(cache, &k, &v);
  if (st == ACP_OK) st = attend_plan(qd, k, b, &P);
  if (st != ACP_OK) return st;
  *bytes = P.workspace;
  return ret(ACP_OK);
}

acp_status cache_attention(const acp_tile_desc* out, const acp_tile_desc* q, const acp_paged_cache* cache,
                           const acp_sequences* b, float scale, void* workspace, int64_t workspace_bytes, void* stream) {
  acp::DescData qd, od;
  CacheSide k, v;
  AttendPlan P;
  acp_status st = load_heads(q, "q", &qd);
  if (st == ACP_OK) st = load_heads(out, "the output", &od);
  if (st == ACP_OK) st = load_cache(cache, &k, &v);
  if (st == ACP_OK) st = check_like(od, qd, true, "the output");
  if (st == ACP_OK) st = attend_plan(qd, k, b, &P);
  if (st != ACP_OK) return st;
  // times log2 e it is a number of float32 still
  if (!(std::fabs(scale) <= 0x1p127f)) return ret(ACP_ERR_INVALID, "the scale is not finite, or past 2^127");
  if (self_overlap(od)) return ret(ACP_ERR_INVALID, "the output overlaps itself");
  if (P.workspace > 0) {
    if (!workspace || workspace_bytes < P.workspace)
      return ret(ACP_ERR_INVALID, "the workspace is smaller than acp_cache_attention_workspace says");
    if (reinterpret_cast<uint64_t>(workspace) % 16) return ret(ACP_ERR_INVALID, "the workspace is not 16-byte aligned");
  }
  const Range w[] = {range_of(od, "the output"), range_of(workspace, P.workspace, "the workspace")};
  Range r[9];
  int nr = 0;
  r[nr++] = range_of(qd, "q");
  r[nr++] = range_of(k.d, "the cache's k");
  r[nr++] = range_of(v.d, "the cache's v");
  if (k.kind != acp::kCacheSame) {
    r[nr++] = range_of(k.scales, cache_scale_bytes(k), "the scales of k");
    r[nr++] = range_of(v.scales, cache_scale_bytes(v), "the scales of v");
  }
  batch_ranges(*b, r, &nr);
  if ((st = check_ranges(w, 2, r, nr)) != ACP_OK) return st;
  acp::AttendArgs& A = P.A;
  acp::HeadsCore core{};
  HeadTensors T;
  T.add(qd, &A.q);
  T.add(od, &A.out);
  if ((st = token_geometry(T, &core)) != ACP_OK) return st;
  A.n2 = core.n2;
  if (P.tokens == 0 || heads_of(qd) == 0 || b->sequences == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  set_cache(k, &A.k);
  set_cache(v, &A.v);
  auto aligned16 = [](const CacheSide& c) {
    bool all = c.d.gbase % 16 == 0;
    for (int d = 0; d < 3; ++d) all = all && (c.d.shape[d] == 1 || c.d.strides[d] * c.d.esize % 16 == 0);
    return all;
  };
  A.direct = k.kind == acp::kCacheSame && aligned16(k) && aligned16(v);
  // zero becomes the least there is, which leaves any score under 2^-21: a weight of
  // what is hidden stays zero
  A.scale = std::max(static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634),
                     std::numeric_limits<float>::denorm_min());
  A.flip = scale < 0.0f ? 0x80008000u : 0u;
  A.part = static_cast<float*>(workspace);
  A.stat = reinterpret_cast<float*>(static_cast<char*>(workspace) + P.stat_at);
  A.joins = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + P.joins_at);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool few = P.tile_rows == acp::kStepRows;
  hipError_t e = few ? acp::attend_step_launch(P.dt, P.cache, P.padded, A, s)
                     : acp::attend_prompt_launch(P.dt, P.cache, P.padded, A, s);
  if (e == hipSuccess && A.shares > 0) e = acp::attend_join_launch(P.dt, P.tile_rows, A, P.join, s);
  return launched(e, std::string("cache attention ") + (few ? "few rows" : "many rows") +
                         (k.kind == acp::kCacheSame ? "" : " 8 bits") + " channels " + std::to_string(P.padded) + " slots " +
                         std::to_string(A.slots.d) + " heads " + std::to_string(1 << A.side_log2) + " shares " +
                         std::to_string(A.shares));
}

}  // namespace

extern "C" {

acp_status acp_cache_attention_workspace(const acp_tile_desc* q, const acp_paged_cache* cache,
                                         const acp_sequences* sequences, int64_t* bytes) {
  return guarded([&] { return cache_attention_workspace(q, cache, sequences, bytes); });
}

acp_status acp_cache_attention(const acp_tile_desc* out, const acp_tile_desc* q, const acp_paged_cache* cache,
                               const acp_sequences* sequences, float scale, void* workspace, int64_t workspace_bytes,
                               void* hip_stream) {
  return guarded(
      [&] { return cache_attention(out, q, cache, sequences, scale, workspace, workspace_bytes, hip_stream); });
}

}  // extern "C"
