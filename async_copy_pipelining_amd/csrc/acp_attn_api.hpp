// Entry points of attention over a paged cache.  Included by acp_entry.cpp
// after acp_heads_api.hpp, whose helpers it uses.
#include "acp_attn.hpp"

namespace {

// Workgroups that a launch aims at where its keys can be split: four for each
// of 256 CUs.
constexpr int64_t kAttendGroups = 1024;
// Keys of a chunk are worth a workgroup of their own from here on.
constexpr int64_t kAttendLeast = 256;
// Rows of a sequence, on average, from which on tiles of 128 rows are taken.
constexpr int64_t kAttendPrompt = 64;

struct AttendPlan {
  acp::AttendArgs A{};
  int tile_rows = 0, padded = 0, cache = 0, dt = 0;
  int64_t workspace = 0, tokens = 0;
  int64_t stat_at = 0;
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
  A.kv_heads = div_by(static_cast<uint64_t>(kv));
  A.heads = div_by(static_cast<uint64_t>(std::max<int64_t>(1, heads)));
  if (P->tokens == 0 || heads == 0 || sequences == 0) return ACP_OK;
  // rows of a sequence: its tokens' query heads of one of the cache's
  const int64_t rows = b->starts ? P->tokens * group : sequences * group;
  P->tile_rows = rows >= kAttendPrompt * sequences ? acp::kPromptRows : acp::kStepRows;
  const int64_t M = P->tile_rows;
  const int64_t slots = b->starts ? P->tokens * group / M + sequences : sequences * ceil_div(group, M);
  if (slots >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 tiles of rows");
  A.slots = div_by(static_cast<uint64_t>(slots));
  // the longest that a sequence can be
  int64_t longest = std::min<int64_t>(int64_t(b->max_pages) * k.d.shape[1], (int64_t(1) << 31) - 1);
  if (b->max_length) longest = std::min<int64_t>(longest, b->max_length);
  longest = std::max<int64_t>(1, longest);
  // sequences mostly fill fewer tiles than their slots
  const int64_t tiles = kv * std::max<int64_t>(sequences, b->starts ? P->tokens * group / M : slots);
  const int64_t wanted = std::max<int64_t>(1, kAttendGroups / tiles);
  int64_t chunk = std::max(ceil_div(longest, wanted), std::min(longest, kAttendLeast));
  chunk = ceil_div(chunk, acp::kChunkUnit) * acp::kChunkUnit;
  const int64_t splits = ceil_div(longest, chunk);
  A.chunk = static_cast<uint32_t>(chunk);
  A.splits = static_cast<uint32_t>(splits);
  // a launch has fewer than 2^32 lanes
  if (kv * slots >= int64_t(1) << 24 || kv * slots * splits >= int64_t(1) << 24 || P->tokens * heads >= int64_t(1) << 26)
    return ret(ACP_ERR_UNSUPPORTED, "a launch of 2^32 lanes");
  P->stat_at = align_up(splits * P->tokens * heads * dim * 4, 16);
  if (splits > 1) P->workspace = P->stat_at + splits * P->tokens * heads * 8;
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
  if (!std::isfinite(scale)) return ret(ACP_ERR_INVALID, "the scale is not finite");
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
  A.scale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  A.part = static_cast<float*>(workspace);
  A.stat = reinterpret_cast<float*>(static_cast<char*>(workspace) + P.stat_at);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool few = P.tile_rows == acp::kStepRows;
  hipError_t e = few ? acp::attend_step_launch(P.dt, P.cache, P.padded, A, s)
                     : acp::attend_prompt_launch(P.dt, P.cache, P.padded, A, s);
  if (e == hipSuccess && A.splits > 1) e = acp::attend_join_launch(P.dt, P.tile_rows, A, s);
  return launched(e, std::string("cache attention ") + (few ? "few rows" : "many rows") +
                         (k.kind == acp::kCacheSame ? "" : " 8 bits") + " channels " + std::to_string(P.padded) + " slots " +
                         std::to_string(A.slots.d) + " splits " + std::to_string(A.splits) + " chunk " +
                         std::to_string(A.chunk));
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
