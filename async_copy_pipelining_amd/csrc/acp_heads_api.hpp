// Entry points of the head operators: rotary positions, head norms, appending
// to a paged cache.  Included by acp_entry.cpp after acp_rows_api.hpp, whose
// helpers it uses.  Host code: checks, the collapse of the token dims, and the
// split of the work; one or two kernels on the caller's stream.
#include "acp_heads.hpp"

namespace {

// Waves that a launch aims at before it gives a wave more than one pass: sixteen
// for each of 256 CUs ([8191, 5 + 1, 80] float32 turned in 11.9 us, with 1024 or
// 8192 waves in 13.6).
constexpr int64_t kHeadWaves = 4096;
// Passes of a wave over its tokens' heads, which share one set of angles (norm of
// [4096, 16 + 4, 128] float16 10.2 us, with 4 of them 11.4).
constexpr int64_t kHeadPasses = 8;
// Workgroups of a backward pass: each leaves 8 bytes a channel ([16384, 32 + 8,
// 128] bfloat16 105 us, with 256 of them 137, with 1024 109).
constexpr int64_t kHeadGradGroups = 512;

bool same_elements_exactly(const acp::DescData& a, const acp::DescData& b) {
  if (a.gbase != b.gbase || a.dtype != b.dtype || !same_shape(a, b)) return false;
  for (int d = 0; d < a.rank; ++d)
    if (a.shape[d] > 1 && a.strides[d] != b.strides[d]) return false;
  return true;
}

// The tensors of one call: all of one type, rank and token dims; tensor k has
// heads[k] heads.
struct HeadTensors {
  const acp::DescData* t[8];
  acp::HeadTensor* out[8];
  int n = 0;
  void add(const acp::DescData& d, acp::HeadTensor* o) {
    t[n] = &d;
    out[n++] = o;
  }
};

int64_t heads_of(const acp::DescData& t) { return t.shape[t.rank - 2]; }
int64_t dim_of(const acp::DescData& t) { return t.shape[t.rank - 1]; }
int64_t tokens_of(const acp::DescData& t) {
  int64_t n = 1;
  for (int d = 0; d + 2 < t.rank; ++d) n *= t.shape[d];
  return n;
}

acp_status load_heads(const acp_tile_desc* d, const char* what, acp::DescData* out) {
  const acp_status st = load_float(d, what, out);
  if (st != ACP_OK) return st;
  if (out->rank < 3) return ret(ACP_ERR_INVALID, std::string(what) + " needs token, head and channel dims");
  return ACP_OK;
}

// As `like` but for the heads.
acp_status check_like(const acp::DescData& t, const acp::DescData& like, bool same_heads, const char* what) {
  bool same = t.rank == like.rank && t.dtype == like.dtype;
  for (int d = 0; same && d < t.rank; ++d)
    same = t.shape[d] == like.shape[d] || (d == t.rank - 2 && !same_heads);
  return same ? ACP_OK : ret(ACP_ERR_INVALID, std::string(what) + " differs in shape or dtype");
}

// Strides of every tensor over the token dims, as at most two dims.
acp_status token_geometry(const HeadTensors& T, acp::HeadsCore* A) {
  const acp::DescData& f = *T.t[0];
  int64_t ext[acp::kMaxInputRank], stride[8][acp::kMaxInputRank];
  int n = 0;
  for (int d = 0; d + 2 < f.rank; ++d) {
    if (f.shape[d] == 1) continue;
    bool join = n > 0;
    for (int k = 0; join && k < T.n; ++k) join = stride[k][n - 1] == f.shape[d] * T.t[k]->strides[d] * T.t[k]->esize;
    if (join) ext[n - 1] *= f.shape[d];
    else ext[n++] = f.shape[d];
    for (int k = 0; k < T.n; ++k) stride[k][n - 1] = T.t[k]->strides[d] * T.t[k]->esize;
  }
  if (n > 2) return ret(ACP_ERR_UNSUPPORTED, "the token dims of these strides do not join into two");
  const int64_t tokens = tokens_of(f);
  if (tokens >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 tokens");
  A->tokens = static_cast<uint32_t>(tokens);
  A->n2 = div_by(static_cast<uint64_t>(n ? std::max<int64_t>(1, ext[n - 1]) : 1));
  for (int k = 0; k < T.n; ++k) {
    const acp::DescData& t = *T.t[k];
    T.out[k]->p = reinterpret_cast<char*>(t.gbase);
    T.out[k]->s[0] = n == 2 ? stride[k][0] : n == 1 ? stride[k][0] * ext[0] : 0;
    T.out[k]->s[1] = n ? stride[k][n - 1] : 0;
    T.out[k]->s[2] = t.strides[t.rank - 2] * t.esize;
  }
  return ACP_OK;
}

acp_status check_rotary(const acp_rotary* r, int64_t dim, acp::HeadsCore* A) {
  A->turn_scale = A->sign = 1.0f;
  if (!r) return ACP_OK;
  if (r->rotated < 2 || r->rotated % 2 || r->rotated > dim)
    return ret(ACP_ERR_INVALID, "the turned channels are an even number from 2 to the head's");
  if (r->layout != ACP_ROTARY_HALVES && r->layout != ACP_ROTARY_PAIRS)
    return ret(ACP_ERR_INVALID, "unknown rotary layout");
  if (!r->frequencies || reinterpret_cast<uint64_t>(r->frequencies) % 8)
    return ret(ACP_ERR_INVALID, "the frequencies need 8-byte aligned float64 values");
  if (!std::isfinite(r->scale)) return ret(ACP_ERR_INVALID, "the rotary scale is not finite");
  A->frequencies = r->frequencies;
  A->rotated = static_cast<uint32_t>(r->rotated);
  A->turn_scale = r->scale;
  return ACP_OK;
}

// A row's units and a wave's lanes; heads[] of up to three sides, whose passes
// are written.
acp_status head_split(int64_t dim, int esize, int pairs, bool one_token, const int64_t* heads, uint32_t** passes,
                      int sides, acp::HeadsCore* A, acp::HeadsShape* K) {
  if (dim < 1) return ret(ACP_ERR_INVALID, "a head needs at least one channel");
  const int64_t v = 16 / esize, half = A->rotated / 2, rest = dim - A->rotated;
  const int64_t turned = ceil_div(half, v), units = turned + ceil_div(rest, 2 * v);
  if (units > 64) return ret(ACP_ERR_UNSUPPORTED, "a head of more than 64 units of 32 bytes");
  A->dim = static_cast<uint32_t>(dim);
  A->turn_units = static_cast<uint32_t>(turned);
  A->units = static_cast<uint32_t>(units);
  K->whole = half % v == 0 && rest % (2 * v) == 0;
  K->pairs = pairs != 0;
  int lanes = 0;
  while ((int64_t(1) << lanes) < units) ++lanes;
  const int rows = 6 - lanes;  // log2 of a wave's rows
  auto total = [&](int log2) {
    int64_t n = 0;
    for (int k = 0; k < sides; ++k) n += ceil_div(heads[k], int64_t(1) << log2);
    return n;
  };
  auto groups = [&](int log2) { return ceil_div(A->tokens, int64_t(1) << (rows - log2)); };
  int hs = one_token ? rows : 0;
  while (hs < rows && (total(hs) > kHeadPasses || groups(hs) * total(hs) < kHeadWaves) && total(hs) > 1) ++hs;
  const int64_t all = std::max<int64_t>(1, total(hs)), g = groups(hs);
  const int64_t shares = std::min(all, std::max<int64_t>(1, kHeadWaves / std::max<int64_t>(1, g)));
  const int64_t each = ceil_div(all, shares), parts = ceil_div(all, each);
  // a launch has fewer than 2^32 lanes
  if (g * parts >= (int64_t(1) << 26) - 4) return ret(ACP_ERR_UNSUPPORTED, "a launch of 2^32 lanes");
  for (int k = 0; k < sides; ++k) *passes[k] = static_cast<uint32_t>(ceil_div(heads[k], int64_t(1) << hs));
  const int64_t rest_units = units - turned;
  A->keep = (turned > 0 && turned < 8) || (rest_units > 0 && rest_units < 8);
  A->lanes_log2 = lanes;
  A->heads_log2 = hs;
  A->groups = static_cast<uint32_t>(g);
  A->per_wave = static_cast<uint32_t>(each);
  A->parts = div_by(static_cast<uint64_t>(parts));
  return ACP_OK;
}

std::string heads_text(const char* what, const acp::HeadsCore& A, const acp::HeadsShape& K) {
  return std::string(what) + (A.rotated ? (K.pairs ? " pairs" : " halves") : "") + (K.whole ? " whole" : " any") +
         " lanes " + std::to_string(1 << A.lanes_log2) + " heads " + std::to_string(1 << A.heads_log2) + " passes " +
         std::to_string(A.per_wave) + " waves " + std::to_string(A.groups * A.parts.d);
}

acp_status check_positions(const int32_t* positions) {
  if (reinterpret_cast<uint64_t>(positions) % 4) return ret(ACP_ERR_INVALID, "the positions are not 4-byte aligned");
  return ACP_OK;
}

// Ranges that the rotation reads.
void rotary_ranges(const acp_rotary* r, const int32_t* positions, int64_t tokens, Range* in, int* n) {
  if (!r) return;
  in[(*n)++] = range_of(r->frequencies, int64_t(r->rotated) * 4, "the frequencies");
  in[(*n)++] = range_of(positions, tokens * 4, "the positions");
}

acp_status heads_forward(const acp_tile_desc* yq, const acp_tile_desc* q, const float* wq, const acp_tile_desc* yk,
                         const acp_tile_desc* k, const float* wk, bool norm, float eps, const int32_t* positions,
                         const acp_rotary* rotary, bool backward, void* stream) {
  acp::DescData x[2], y[2];
  acp_status st = load_heads(q, "q", &x[0]);
  if (st == ACP_OK) st = load_heads(yq, "the turned q", &y[0]);
  if (st != ACP_OK) return st;
  if ((k != nullptr) != (yk != nullptr)) return ret(ACP_ERR_INVALID, "k and its output are given together or not at all");
  if (k && (st = load_heads(k, "k", &x[1])) != ACP_OK) return st;
  if (k && (st = load_heads(yk, "the turned k", &y[1])) != ACP_OK) return st;
  const int sides = k ? 2 : 1;
  if ((st = check_like(y[0], x[0], true, "q's output")) != ACP_OK) return st;
  if (k && (st = check_like(x[1], x[0], false, "k")) != ACP_OK) return st;
  if (k && (st = check_like(y[1], x[1], true, "k's output")) != ACP_OK) return st;
  if (norm && (!(eps >= 0.0f) || std::isinf(eps))) return ret(ACP_ERR_INVALID, "eps must be a finite number >= 0");
  if (misaligned4(wq) || misaligned4(wk)) return ret(ACP_ERR_INVALID, "a float32 array is not 4-byte aligned");
  if ((st = check_positions(positions)) != ACP_OK) return st;
  acp::HeadsForward A{};
  acp::HeadsShape K{};
  const int64_t dim = dim_of(x[0]);
  if (!norm && !rotary) return ret(ACP_ERR_INVALID, "a rotation needs its frequencies");
  if ((st = check_rotary(rotary, dim, &A)) != ACP_OK) return st;
  HeadTensors T;
  int64_t heads[2] = {};
  uint32_t* passes[2] = {&A.side[0].passes, &A.side[1].passes};
  Range w[2], r[8];
  int nw = 0, nr = 0;
  for (int s = 0; s < sides; ++s) {
    static const char* const names[2][2] = {{"q", "q's output"}, {"k", "k's output"}};
    if (self_overlap(y[s])) return ret(ACP_ERR_INVALID, "an output overlaps itself");
    T.add(x[s], &A.side[s].x);
    T.add(y[s], &A.side[s].y);
    heads[s] = heads_of(x[s]);
    A.side[s].heads = static_cast<uint32_t>(heads[s]);
    A.side[s].weight = s ? wk : wq;
    w[nw++] = range_of(y[s], names[s][1]);
    // in place: a lane has read a row before it writes there
    if (!same_elements_exactly(x[s], y[s])) r[nr++] = range_of(x[s], names[s][0]);
    r[nr++] = range_of(A.side[s].weight, dim * 4, s ? "wk" : "wq");
    if (heads[s] >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 heads");
  }
  const int64_t tokens = tokens_of(x[0]);
  rotary_ranges(rotary, positions, tokens, r, &nr);
  if ((st = check_ranges(w, nw, r, nr)) != ACP_OK) return st;
  if ((st = token_geometry(T, &A)) != ACP_OK) return st;
  if ((st = head_split(dim, x[0].esize, rotary && rotary->layout == ACP_ROTARY_PAIRS, false, heads, passes, sides, &A, &K)) !=
      ACP_OK)
    return st;
  if (tokens == 0 || heads[0] + heads[1] == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  A.positions = positions;
  A.span = div_by(static_cast<uint64_t>(x[0].shape[x[0].rank - 3]));
  A.sign = backward ? -1.0f : 1.0f;
  A.eps = eps;
  K.dt = row_dtype(x[0].dtype);
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  return launched(norm ? acp::head_norm_launch(K, A, hs) : acp::rotate_launch(K, A, hs),
                  heads_text(norm ? "head norm" : backward ? "rotate back" : "rotate", A, K));
}

int64_t head_grad_groups(int64_t tokens, int64_t heads) {
  return std::max<int64_t>(1, std::min(kHeadGradGroups, ceil_div(tokens * heads, acp::kHeadThreads / 64)));
}

acp_status head_norm_workspace(const acp_tile_desc* q, const acp_tile_desc* k, int64_t* bytes) {
  acp::DescData x[2];
  if (!bytes) return ret(ACP_ERR_INVALID, "null argument");
  acp_status st = load_heads(q, "q", &x[0]);
  if (st == ACP_OK && k) st = load_heads(k, "k", &x[1]);
  if (st == ACP_OK && k) st = check_like(x[1], x[0], false, "k");
  if (st != ACP_OK) return st;
  const int64_t tokens = tokens_of(x[0]), heads = heads_of(x[0]) + (k ? heads_of(x[1]) : 0);
  if (tokens >= kRowLimit || heads >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 tokens or heads");
  *bytes = head_grad_groups(tokens, heads) * 2 * dim_of(x[0]) * 4;
  return ret(ACP_OK);
}

acp_status head_norm_backward(const acp_tile_desc* dq, float* dwq, const acp_tile_desc* dyq, const acp_tile_desc* q,
                              const float* wq, const acp_tile_desc* dk, float* dwk, const acp_tile_desc* dyk,
                              const acp_tile_desc* k, const float* wk, float eps, const int32_t* positions,
                              const acp_rotary* rotary, void* workspace, int64_t workspace_bytes, void* stream) {
  acp::DescData x[2], dy[2], dx[2];
  if ((k != nullptr) != (dk != nullptr) || (k != nullptr) != (dyk != nullptr))
    return ret(ACP_ERR_INVALID, "k and its gradients are given together or not at all");
  if (!k && (dwk || wk)) return ret(ACP_ERR_INVALID, "a weight of k without k");
  const int sides = k ? 2 : 1;
  acp_status st = ACP_OK;
  for (int s = 0; s < sides && st == ACP_OK; ++s) {
    st = load_heads(s ? k : q, s ? "k" : "q", &x[s]);
    if (st == ACP_OK) st = load_heads(s ? dyk : dyq, s ? "dyk" : "dyq", &dy[s]);
    if (st == ACP_OK) st = load_heads(s ? dk : dq, s ? "dk" : "dq", &dx[s]);
    if (st == ACP_OK) st = check_like(x[s], x[0], s == 0, "k");
    if (st == ACP_OK) st = check_like(dy[s], x[s], true, "a gradient");
    if (st == ACP_OK) st = check_like(dx[s], x[s], true, "a gradient");
  }
  if (st != ACP_OK) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return ret(ACP_ERR_INVALID, "eps must be a finite number >= 0");
  if (misaligned4(wq) || misaligned4(wk) || misaligned4(dwq) || misaligned4(dwk))
    return ret(ACP_ERR_INVALID, "a float32 array is not 4-byte aligned");
  if ((st = check_positions(positions)) != ACP_OK) return st;
  acp::HeadsBackward A{};
  acp::HeadsShape K{};
  const int64_t dim = dim_of(x[0]);
  if ((st = check_rotary(rotary, dim, &A)) != ACP_OK) return st;
  const int64_t tokens = tokens_of(x[0]);
  int64_t heads[2] = {heads_of(x[0]), k ? heads_of(x[1]) : 0};
  if (heads[0] >= kRowLimit || heads[1] >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 heads");
  const bool sums = dwq || dwk;
  HeadTensors T;
  uint32_t* passes[2] = {&A.side[0].passes, &A.side[1].passes};
  for (int s = 0; s < sides; ++s) {
    if (self_overlap(dx[s])) return ret(ACP_ERR_INVALID, "an output overlaps itself");
    T.add(x[s], &A.side[s].x);
    T.add(dy[s], &A.side[s].dy);
    T.add(dx[s], &A.side[s].dx);
    A.side[s].heads = static_cast<uint32_t>(heads[s]);
    A.side[s].weight = s ? wk : wq;
  }
  if ((st = token_geometry(T, &A)) != ACP_OK) return st;
  if ((st = head_split(dim, x[0].esize, rotary && rotary->layout == ACP_ROTARY_PAIRS, false, heads, passes, sides, &A, &K)) !=
      ACP_OK)
    return st;
  const int64_t items = int64_t(A.groups) * A.parts.d;
  const int64_t groups = std::min(head_grad_groups(tokens, heads[0] + heads[1]), std::max<int64_t>(1, ceil_div(items, 4)));
  const int64_t need = sums && tokens > 0 ? groups * 2 * dim * 4 : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return ret(ACP_ERR_INVALID, "the workspace is smaller than acp_head_norm_workspace says");
    if (reinterpret_cast<uint64_t>(workspace) % 16) return ret(ACP_ERR_INVALID, "the workspace is not 16-byte aligned");
  }
  Range w[5], r[12];
  int nw = 0, nr = 0;
  for (int s = 0; s < sides; ++s) {
    w[nw++] = range_of(dx[s], s ? "dk" : "dq");
    w[nw++] = range_of(s ? dwk : dwq, dim * 4, s ? "dwk" : "dwq");
    // in place: a lane has read a row before it writes there
    if (!same_elements_exactly(x[s], dx[s])) r[nr++] = range_of(x[s], s ? "k" : "q");
    if (!same_elements_exactly(dy[s], dx[s])) r[nr++] = range_of(dy[s], s ? "dyk" : "dyq");
    r[nr++] = range_of(A.side[s].weight, dim * 4, s ? "wk" : "wq");
  }
  w[nw++] = range_of(workspace, need, "the workspace");
  rotary_ranges(rotary, positions, tokens, r, &nr);
  if ((st = check_ranges(w, nw, r, nr)) != ACP_OK) return st;
  if ((st = check_stream(stream)) != ACP_OK) return st;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  acp::HeadColumns C{};
  C.part = static_cast<const float*>(workspace);
  C.out[0] = dwq;
  C.out[1] = dwk;
  C.dim = static_cast<uint32_t>(dim);
  C.pitch = static_cast<uint32_t>(2 * dim);
  if (tokens == 0 || heads[0] + heads[1] == 0) {  // the gradients of the weights are zero
    if (!sums) return launched_nothing();
    return launched(acp::head_columns_launch(C, hs), "head norm backward of no tokens");
  }
  A.positions = positions;
  A.span = div_by(static_cast<uint64_t>(x[0].shape[x[0].rank - 3]));
  A.sign = -1.0f;
  A.eps = eps;
  A.part_pitch = C.pitch;
  A.side[0].part = dwq ? static_cast<float*>(workspace) : nullptr;
  A.side[1].part = dwk ? static_cast<float*>(workspace) + dim : nullptr;
  K.dt = row_dtype(x[0].dtype);
  hipError_t e = acp::head_norm_backward_launch(K, A, static_cast<uint32_t>(groups), hs);
  C.rows = static_cast<uint32_t>(groups);
  if (e == hipSuccess && sums) e = acp::head_columns_launch(C, hs);
  return launched(e, heads_text("head norm backward", A, K) + " workgroups " + std::to_string(groups));
}

// Frequencies of the turned pairs, on the host.
acp_status rotary_frequencies(double* out, int rotated, double base, acp_rotary_scaling scaling, double factor,
                              double length, double low, double high) {
  if (!out) return ret(ACP_ERR_INVALID, "null argument");
  if (rotated < 2 || rotated % 2) return ret(ACP_ERR_INVALID, "the turned channels are an even number from 2 on");
  if (!(base > 0.0) || std::isinf(base)) return ret(ACP_ERR_INVALID, "the base must be a finite number > 0");
  if (scaling != ACP_ROTARY_PLAIN && scaling != ACP_ROTARY_LINEAR && scaling != ACP_ROTARY_BASE &&
      scaling != ACP_ROTARY_BANDS)
    return ret(ACP_ERR_INVALID, "unknown rotary scaling");
  if (scaling != ACP_ROTARY_PLAIN && (!(factor >= 1.0) || std::isinf(factor)))
    return ret(ACP_ERR_INVALID, "the factor must be a finite number >= 1");
  if (scaling == ACP_ROTARY_BASE && rotated < 4)
    return ret(ACP_ERR_INVALID, "a scaled base needs at least two pairs");
  if (scaling == ACP_ROTARY_BANDS &&
      (!(length > 0.0) || std::isinf(length) || !(low >= 0.0) || !(high > low) || std::isinf(high)))
    return ret(ACP_ERR_INVALID, "bands need a length > 0 and 0 <= low < high turns");
  constexpr double kTwoPi = 6.283185307179586476925;
  if (scaling == ACP_ROTARY_BASE) base *= std::pow(factor, rotated / (rotated - 2.0));
  for (int i = 0; i < rotated / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rotated);
    if (scaling == ACP_ROTARY_LINEAR) f /= factor;
    if (scaling == ACP_ROTARY_BANDS) {
      const double keep = std::min(1.0, std::max(0.0, (length * f / kTwoPi - low) / (high - low)));
      f *= keep + (1.0 - keep) / factor;
    }
    out[i] = f;
  }
  return ret(ACP_OK);
}

// ---------------------------------------------------------------- paged caches

// A cache's keys or values: [pages, page, heads, dim].
struct CacheSide {
  acp::DescData d;
  float* scales = nullptr;
  int kind = acp::kCacheSame;
};

acp_status load_cache_side(const acp_tile_desc* plain, const acp_packed8* packed, const char* what, CacheSide* out) {
  if ((plain != nullptr) == (packed != nullptr))
    return ret(ACP_ERR_INVALID, std::string(what) + " has a descriptor or an 8-bit form, and not both");
  if (plain) {
    const acp_status st = load_float(plain, what, &out->d);
    if (st != ACP_OK) return st;
  } else {
    if (!load_desc(packed->codes, &out->d))
      return ret(ACP_ERR_INVALID, std::string(what) + " has no encoded descriptor of its codes");
    const acp_status st = load_packed(packed, out->d, what, &out->d);
    if (st != ACP_OK) return st;
    out->scales = packed->scales;
    out->kind = packed->format == ACP_PACK_I8 ? acp::kCacheI8 : acp::kCacheE4M3;
  }
  if (out->d.rank != 4) return ret(ACP_ERR_INVALID, std::string(what) + " is [pages, positions, heads, channels]");
  if (packed && packed->block < out->d.shape[3])
    return ret(ACP_ERR_UNSUPPORTED, std::string(what) + " has one scale a row: a block of at least its channels");
  for (int k = 0; k < 3; ++k)
    if (out->d.shape[k] >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, std::string(what) + " has 2^31 pages, positions or heads");
  if (out->d.shape[1] < 1) return ret(ACP_ERR_INVALID, "a page holds at least one position");
  if (self_overlap(out->d)) return ret(ACP_ERR_INVALID, std::string(what) + " overlaps itself");
  return ACP_OK;
}

acp_status load_cache(const acp_paged_cache* c, CacheSide* k, CacheSide* v) {
  if (!c) return ret(ACP_ERR_INVALID, "no cache");
  acp_status st = load_cache_side(c->k, c->k8, "the cache's k", k);
  if (st == ACP_OK) st = load_cache_side(c->v, c->v8, "the cache's v", v);
  if (st != ACP_OK) return st;
  if (!same_shape(k->d, v->d) || k->d.dtype != v->d.dtype || k->kind != v->kind)
    return ret(ACP_ERR_INVALID, "the cache's k and v differ in shape, dtype or format");
  return ACP_OK;
}

acp_status load_batch(const acp_sequences* b, const CacheSide& k, acp::BatchArgs* out) {
  if (!b) return ret(ACP_ERR_INVALID, "no sequences");
  if (b->sequences < 0 || b->max_pages < 0 || b->max_length < 0)
    return ret(ACP_ERR_INVALID, "a negative number of sequences, pages or positions");
  if (b->sequences > 0 && (!b->lengths || (b->max_pages > 0 && !b->pages)))
    return ret(ACP_ERR_INVALID, "the sequences need their lengths and pages");
  for (const int32_t* p : {b->starts, b->lengths, b->pages})
    if (reinterpret_cast<uint64_t>(p) % 4) return ret(ACP_ERR_INVALID, "an int32 array is not 4-byte aligned");
  out->starts = b->starts;
  out->lengths = b->lengths;
  out->pages = b->pages;
  out->sequences = static_cast<uint32_t>(b->sequences);
  out->max_pages = static_cast<uint32_t>(b->max_pages);
  out->page = div_by(static_cast<uint64_t>(k.d.shape[1]));
  out->page_count = static_cast<uint32_t>(k.d.shape[0]);
  return ACP_OK;
}

void batch_ranges(const acp_sequences& b, Range* r, int* n) {
  r[(*n)++] = range_of(b.starts, (int64_t(b.sequences) + 1) * 4, "the starts");
  r[(*n)++] = range_of(b.lengths, int64_t(b.sequences) * 4, "the lengths");
  r[(*n)++] = range_of(b.pages, int64_t(b.sequences) * b.max_pages * 4, "the pages");
}

int64_t cache_scale_bytes(const CacheSide& c) { return c.d.shape[0] * c.d.shape[1] * c.d.shape[2] * 4; }

void set_cache(const CacheSide& c, acp::CacheTensor* out) {
  out->p = reinterpret_cast<char*>(c.d.gbase);
  for (int k = 0; k < 3; ++k) out->s[k] = c.d.strides[k] * c.d.esize;
  out->scales = c.scales;
}

acp_status cache_append(const acp_paged_cache* cache, const acp_tile_desc* k, const acp_tile_desc* v,
                        const acp_sequences* batch, const acp_rotary* rotary, const acp_tile_desc* yq,
                        const acp_tile_desc* q, void* stream) {
  acp::DescData kd, vd, qd, yd;
  CacheSide ck, cv;
  acp::AppendArgs A{};
  acp_status st = load_cache(cache, &ck, &cv);
  if (st == ACP_OK) st = load_heads(k, "k", &kd);
  if (st == ACP_OK) st = load_heads(v, "v", &vd);
  if (st != ACP_OK) return st;
  if ((q != nullptr) != (yq != nullptr)) return ret(ACP_ERR_INVALID, "q and its output are given together or not at all");
  if ((st = check_like(vd, kd, true, "v")) != ACP_OK) return st;
  if (q) {
    if ((st = load_heads(q, "q", &qd)) != ACP_OK) return st;
    if ((st = load_heads(yq, "the turned q", &yd)) != ACP_OK) return st;
    if ((st = check_like(qd, kd, false, "q")) != ACP_OK) return st;
    if ((st = check_like(yd, qd, true, "q's output")) != ACP_OK) return st;
    if (self_overlap(yd)) return ret(ACP_ERR_INVALID, "an output overlaps itself");
    if (heads_of(qd) >= kRowLimit) return ret(ACP_ERR_UNSUPPORTED, "2^31 heads");
  }
  if (heads_of(kd) != ck.d.shape[2] || dim_of(kd) != ck.d.shape[3])
    return ret(ACP_ERR_INVALID, "the new rows and the cache's differ in heads or channels");
  if (ck.kind == acp::kCacheSame && ck.d.dtype != kd.dtype)
    return ret(ACP_ERR_INVALID, "the new rows and the cache's differ in dtype");
  if ((st = load_batch(batch, ck, &A.batch)) != ACP_OK) return st;
  const int64_t dim = dim_of(kd), tokens = tokens_of(kd);
  if ((st = check_rotary(rotary, dim, &A)) != ACP_OK) return st;
  HeadTensors T;
  T.add(kd, &A.k.x);
  T.add(vd, &A.v.x);
  if (q) {
    T.add(qd, &A.q.x);
    T.add(yd, &A.q.y);
  }
  Range w[5], r[9];
  int nw = 0, nr = 0;
  w[nw++] = range_of(ck.d, "the cache's k");
  w[nw++] = range_of(cv.d, "the cache's v");
  if (ck.kind != acp::kCacheSame) {
    w[nw++] = range_of(ck.scales, cache_scale_bytes(ck), "the scales of k");
    w[nw++] = range_of(cv.scales, cache_scale_bytes(cv), "the scales of v");
  }
  r[nr++] = range_of(kd, "k");
  r[nr++] = range_of(vd, "v");
  if (q) {
    w[nw++] = range_of(yd, "q's output");
    // in place: a lane has read a row before it writes there
    if (!same_elements_exactly(qd, yd)) r[nr++] = range_of(qd, "q");
  }
  rotary_ranges(rotary, nullptr, 0, r, &nr);
  batch_ranges(*batch, r, &nr);
  if ((st = check_ranges(w, nw, r, nr)) != ACP_OK) return st;
  if ((st = token_geometry(T, &A)) != ACP_OK) return st;
  const int64_t heads[3] = {q ? heads_of(qd) : 0, heads_of(kd), heads_of(kd)};
  uint32_t* passes[3] = {&A.q.passes, &A.k.passes, &A.v.passes};
  acp::HeadsShape K{};
  if ((st = head_split(dim, kd.esize, rotary && rotary->layout == ACP_ROTARY_PAIRS, true, heads, passes, 3, &A, &K)) != ACP_OK)
    return st;
  if (tokens == 0 || batch->sequences == 0 || heads[0] + heads[1] == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  A.q.heads = static_cast<uint32_t>(heads[0]);
  A.k.heads = A.v.heads = static_cast<uint32_t>(heads[1]);
  set_cache(ck, &A.ck);
  set_cache(cv, &A.cv);
  A.format = ck.kind == acp::kCacheE4M3 ? ACP_PACK_E4M3 : ACP_PACK_I8;
  K.dt = row_dtype(kd.dtype);
  return launched(acp::append_launch(K, ck.kind, A, static_cast<hipStream_t>(stream)),
                  heads_text(ck.kind == acp::kCacheSame ? "cache append" : "cache append in 8 bits", A, K));
}

}  // namespace

extern "C" {

acp_status acp_rotary_frequencies(double* frequencies, int rotated, double base, acp_rotary_scaling scaling,
                                  double factor, double length, double low, double high) {
  return guarded([&] { return rotary_frequencies(frequencies, rotated, base, scaling, factor, length, low, high); });
}

acp_status acp_rotate(const acp_tile_desc* yq, const acp_tile_desc* q, const acp_tile_desc* yk, const acp_tile_desc* k,
                      const int32_t* positions, const acp_rotary* rotary, int backward, void* hip_stream) {
  return guarded([&] {
    return heads_forward(yq, q, nullptr, yk, k, nullptr, false, 0.0f, positions, rotary, backward != 0, hip_stream);
  });
}

acp_status acp_head_norm(const acp_tile_desc* yq, const acp_tile_desc* q, const float* wq, const acp_tile_desc* yk,
                         const acp_tile_desc* k, const float* wk, float eps, const int32_t* positions,
                         const acp_rotary* rotary, void* hip_stream) {
  return guarded(
      [&] { return heads_forward(yq, q, wq, yk, k, wk, true, eps, positions, rotary, false, hip_stream); });
}

acp_status acp_head_norm_workspace(const acp_tile_desc* q, const acp_tile_desc* k, int64_t* bytes) {
  return guarded([&] { return head_norm_workspace(q, k, bytes); });
}

acp_status acp_head_norm_backward(const acp_tile_desc* dq, float* dwq, const acp_tile_desc* dyq,
                                  const acp_tile_desc* q, const float* wq, const acp_tile_desc* dk, float* dwk,
                                  const acp_tile_desc* dyk, const acp_tile_desc* k, const float* wk, float eps,
                                  const int32_t* positions, const acp_rotary* rotary, void* workspace,
                                  int64_t workspace_bytes, void* hip_stream) {
  return guarded([&] {
    return head_norm_backward(dq, dwq, dyq, q, wq, dk, dwk, dyk, k, wk, eps, positions, rotary, workspace,
                              workspace_bytes, hip_stream);
  });
}

acp_status acp_cache_append(const acp_paged_cache* cache, const acp_tile_desc* k, const acp_tile_desc* v,
                            const acp_sequences* batch, const acp_rotary* rotary, const acp_tile_desc* yq,
                            const acp_tile_desc* q, void* hip_stream) {
  return guarded([&] { return cache_append(cache, k, v, batch, rotary, yq, q, hip_stream); });
}

}  // extern "C"
