// Entry points of the row operators: 8-bit checkpoints, activations, group
// norm.  Included by acp_entry.cpp after acp_api.cpp, whose helpers it uses.
// Host code: checks, the collapse of the tensors' outer dims, and the split of
// the work; one or two kernels on the caller's stream.
#include <algorithm>
#include <cmath>

#include "acp_rows.hpp"

namespace {

int row_dtype(int dtype) {
  return dtype == ACP_F16 ? acp::kRowF16 : dtype == ACP_BF16 ? acp::kRowBF16 : dtype == ACP_F32 ? acp::kRowF32 : -1;
}

acp::Div div_by(uint64_t d) {
  acp::Div r;
  r.d = static_cast<uint32_t>(d);
  acp::magic_for(r.d, &r.mag, &r.sh);
  return r;
}

bool same_shape(const acp::DescData& a, const acp::DescData& b) {
  if (a.rank != b.rank) return false;
  for (int d = 0; d < a.rank; ++d)
    if (a.shape[d] != b.shape[d]) return false;
  return true;
}

// Whether two elements of a tensor lie at one address.  Taken from the
// strides in ascending order, each has to reach past everything inside it.
bool self_overlap(const acp::DescData& t) {
  int order[acp::kMaxInputRank];
  int n = 0;
  for (int d = 0; d < t.rank; ++d)
    if (t.shape[d] > 1) order[n++] = d;
  std::sort(order, order + n, [&](int a, int b) { return t.strides[a] < t.strides[b]; });
  uint64_t span = 0;
  for (int k = 0; k < n; ++k) {
    if (static_cast<uint64_t>(t.strides[order[k]]) <= span) return true;
    span += static_cast<uint64_t>(t.shape[order[k]] - 1) * static_cast<uint64_t>(t.strides[order[k]]);
  }
  return false;
}

int64_t elements(const acp::DescData& t) {
  int64_t n = 1;
  for (int d = 0; d < t.rank; ++d) n *= t.shape[d];
  return n;
}

// A byte range that a call reads or writes, and the tensor that it belongs to.
struct Range {
  uint64_t at, bytes;
  const char* what;
  const acp::DescData* tensor;
};

Range range_of(const acp::DescData& t, const char* what) { return {t.gbase, tensor_span(t), what, &t}; }
Range range_of(const void* p, int64_t bytes, const char* what) {
  return {reinterpret_cast<uint64_t>(p), p ? static_cast<uint64_t>(bytes) : 0u, what, nullptr};
}

// Whether two tensors lie side by side in one buffer: taken as blocks of their
// dims [k, rank), which repeat at equal strides of the dims before, all a
// multiple of one pitch, each tensor's blocks in their own part of it.  k the
// innermost dim: rows, as the halves of a fused projection; fewer dims before:
// stacked tensors, as [:, 0] and [:, 1] of [batch, 2, ...].
bool side_by_side(const acp::DescData& a, const acp::DescData& b, int k) {
  uint64_t pitch = 0;
  for (int d = 0; d < k; ++d) {
    if (a.shape[d] != b.shape[d]) return false;
    if (a.shape[d] == 1) continue;
    const uint64_t s = static_cast<uint64_t>(a.strides[d]) * a.esize;
    if (s != static_cast<uint64_t>(b.strides[d]) * b.esize) return false;
    pitch = pitch == 0 || s < pitch ? s : pitch;
  }
  if (pitch == 0) return false;
  for (int d = 0; d < k; ++d)
    if (a.shape[d] > 1 && static_cast<uint64_t>(a.strides[d]) * a.esize % pitch) return false;
  auto block = [k](const acp::DescData& t) {
    uint64_t n = t.esize;
    for (int d = k; d < t.rank; ++d)
      n += static_cast<uint64_t>(t.shape[d] - 1) * static_cast<uint64_t>(t.strides[d]) * t.esize;
    return n;
  };
  const uint64_t from =
      b.gbase >= a.gbase ? (b.gbase - a.gbase) % pitch : (pitch - (a.gbase - b.gbase) % pitch) % pitch;
  return from >= block(a) && from + block(b) <= pitch;
}

bool side_by_side(const acp::DescData& a, const acp::DescData& b) {
  if (a.rank != b.rank) return false;
  for (int k = a.rank - 1; k > 0; --k)
    if (side_by_side(a, b, k)) return true;
  return false;
}

bool meet(const Range& a, const Range& b) {
  return overlap(a.at, a.bytes, b.at, b.bytes) && !(a.tensor && b.tensor && side_by_side(*a.tensor, *b.tensor));
}

// Written ranges share no byte with each other or with what is read.
acp_status check_ranges(const Range* out, int n_out, const Range* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (meet(out[i], out[j]))
        return ret(ACP_ERR_INVALID, std::string(out[i].what) + " and " + out[j].what + " share memory");
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i], in[j]))
        return ret(ACP_ERR_INVALID, std::string(out[i].what) + " and " + in[j].what + " share memory");
  }
  return ACP_OK;
}

// A float tensor of a row operator.
acp_status load_float(const acp_tile_desc* d, const char* what, acp::DescData* out) {
  if (!load_desc(d, out)) return ret(ACP_ERR_INVALID, std::string(what) + " is not an encoded descriptor");
  if (row_dtype(out->dtype) < 0) return ret(ACP_ERR_UNSUPPORTED, std::string(what) + " must be f16, bf16 or f32");
  if (out->gbase % out->esize) return ret(ACP_ERR_INVALID, std::string(what) + " is not aligned to its element");
  return ACP_OK;
}

acp_status load_packed(const acp_packed8* p, const acp::DescData& like, const char* what, acp::DescData* out) {
  if (!p || !load_desc(p->codes, out))
    return ret(ACP_ERR_INVALID, std::string(what) + " has no encoded descriptor of its codes");
  if (out->dtype != ACP_U8) return ret(ACP_ERR_INVALID, std::string(what) + " holds u8 codes");
  if (!p->scales || reinterpret_cast<uint64_t>(p->scales) % 4)
    return ret(ACP_ERR_INVALID, std::string(what) + " needs 4-byte aligned scales");
  if (p->format != ACP_PACK_I8 && p->format != ACP_PACK_E4M3)
    return ret(ACP_ERR_INVALID, std::string(what) + " has an unknown 8-bit format");
  if (p->block != 32 && p->block != 64 && p->block != 128 && p->block != 256)
    return ret(ACP_ERR_INVALID, std::string(what) + " needs a block of 32, 64, 128 or 256");
  if (!same_shape(*out, like)) return ret(ACP_ERR_INVALID, std::string(what) + " has another shape");
  return ACP_OK;
}

int64_t scale_bytes(const acp::DescData& codes, int block) {
  const int64_t c = codes.shape[codes.rank - 1];
  return c ? elements(codes) / c * ((c + block - 1) / block) * 4 : 0;
}

// The outer dims [lo, rank - 1) of tensors of one shape as at most `most`
// dims, outermost first: dims that all tensors hold without a gap become one.
struct Collapsed {
  int n = 0;
  int64_t ext[acp::kMaxInputRank];
  int64_t stride[8][acp::kMaxInputRank];  // bytes, by tensor
};

bool collapse(const acp::DescData* const* t, int nt, int lo, int most, Collapsed* out) {
  const int r = t[0]->rank;
  for (int d = lo; d + 1 < r; ++d) {
    if (t[0]->shape[d] == 1) continue;
    bool join = out->n > 0;
    for (int k = 0; join && k < nt; ++k)
      join = out->stride[k][out->n - 1] == t[k]->shape[d] * t[k]->strides[d] * t[k]->esize;
    if (join) out->ext[out->n - 1] *= t[0]->shape[d];
    else out->ext[out->n++] = t[0]->shape[d];
    for (int k = 0; k < nt; ++k) out->stride[k][out->n - 1] = t[k]->strides[d] * t[k]->esize;
  }
  return out->n <= most;
}

int log2_of(int64_t v) { return log2i(static_cast<int>(v)); }

constexpr int64_t kRowLimit = (int64_t(1) << 31) - 4096;  // rows and chunks the kernels index

// Elementwise row operators: the geometry of `t` (all of one shape) in chunks
// of v channels, scale blocks of `block` channels (0: none).  Rows that all
// tensors hold without a gap, in whole scale blocks, become one long row.
acp_status row_geometry(const acp::DescData* const* t, acp::RowTensor* const* rt, int nt, int v, int block,
                        acp::RowsArgs* A) {
  const int r = t[0]->rank;
  Collapsed o;
  if (!collapse(t, nt, 0, 3, &o))
    return ret(ACP_ERR_UNSUPPORTED, "the outer dims of these strides do not join into three");
  const int unit = block ? block : v;
  int64_t c = t[0]->shape[r - 1], rows = 1;
  for (int d = 0; d < o.n; ++d) rows *= o.ext[d];
  bool flat = o.n == 1 && c % unit == 0;
  for (int k = 0; flat && k < nt; ++k) flat = o.stride[k][0] == c * t[k]->esize;
  if (flat) {
    c *= rows;
    rows = 1;
    o.n = 0;
  }
  const int64_t cpr = (c + unit - 1) / unit * (unit / v);
  if (rows >= kRowLimit || cpr >= kRowLimit || rows * cpr >= kRowLimit)
    return ret(ACP_ERR_UNSUPPORTED, "more than 2^31 chunks of 16 bytes");
  const int64_t n1 = o.n >= 2 ? o.ext[o.n - 2] : 1, n2 = o.n >= 1 ? o.ext[o.n - 1] : 1;
  A->c = c;
  A->total = static_cast<uint32_t>(rows * cpr);
  A->cpr = div_by(static_cast<uint64_t>(cpr));
  A->n1 = div_by(static_cast<uint64_t>(n1));
  A->n2 = div_by(static_cast<uint64_t>(n2));
  A->lb_log2 = log2_of(unit / v);
  for (int k = 0; k < nt; ++k) {
    rt[k]->p = reinterpret_cast<char*>(t[k]->gbase);
    for (int d = 0; d < 3; ++d) rt[k]->s[d] = 0;
    for (int d = 0; d < o.n; ++d) rt[k]->s[3 - o.n + d] = o.stride[k][d];
  }
  return ACP_OK;
}

// The kernels run on the current device: a stream of another one is refused.
acp_status check_stream(void* stream) {
  hipDevice_t dev = 0;
  if (stream && hipStreamGetDevice(static_cast<hipStream_t>(stream), &dev) == hipSuccess && dev != current_device())
    return ret(ACP_ERR_INVALID, "the stream is of another device than the current one");
  return ACP_OK;
}

acp_status launched(hipError_t e, const std::string& what) {
  if (e != hipSuccess) {
    g_last_kernel = "none";
    return ret(ACP_ERR_HIP, std::string("kernel launch failed: ") + hipGetErrorString(e));
  }
  g_last_kernel = what;
  return ret(ACP_OK);
}

acp_status launched_nothing() {
  g_last_kernel = "none";
  return ret(ACP_OK);
}

bool known_act(int act) { return act == ACP_ACT_NONE || act == ACP_ACT_SILU || act == ACP_ACT_GELU; }

acp_status pack8(const acp_packed8* out, const acp_tile_desc* x, void* stream) {
  acp::DescData xd, cd;
  acp_status st = load_float(x, "x", &xd);
  if (st == ACP_OK) st = load_packed(out, xd, "the packed output", &cd);
  if (st != ACP_OK) return st;
  if (self_overlap(cd)) return ret(ACP_ERR_INVALID, "the codes overlap themselves");
  const Range w[] = {range_of(cd, "the codes"), range_of(out->scales, scale_bytes(cd, out->block), "the scales")};
  const Range r[] = {range_of(xd, "x")};
  if ((st = check_ranges(w, 2, r, 1)) != ACP_OK) return st;
  if (elements(xd) == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  acp::RowsArgs A{};
  const acp::DescData* t[] = {&xd, &cd};
  acp::RowTensor* rt[] = {&A.x, &A.px.codes};
  const int v = 16 / xd.esize;
  if ((st = row_geometry(t, rt, 2, v, out->block, &A)) != ACP_OK) return st;
  A.px.scales = out->scales;
  A.format = out->format;
  return launched(acp::pack8_launch(row_dtype(xd.dtype), A, static_cast<hipStream_t>(stream)),
                  "pack8 chunks " + std::to_string(A.total));
}

acp_status unpack8(const acp_tile_desc* out, const acp_packed8* in, void* stream) {
  acp::DescData od, cd;
  acp_status st = load_float(out, "the output", &od);
  if (st == ACP_OK) st = load_packed(in, od, "the packed input", &cd);
  if (st != ACP_OK) return st;
  if (self_overlap(od)) return ret(ACP_ERR_INVALID, "the output overlaps itself");
  const Range w[] = {range_of(od, "the output")};
  const Range r[] = {range_of(cd, "the codes"), range_of(in->scales, scale_bytes(cd, in->block), "the scales")};
  if ((st = check_ranges(w, 1, r, 2)) != ACP_OK) return st;
  if (elements(od) == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  acp::RowsArgs A{};
  const acp::DescData* t[] = {&od, &cd};
  acp::RowTensor* rt[] = {&A.y, &A.px.codes};
  const int v = 16 / od.esize;
  if ((st = row_geometry(t, rt, 2, v, in->block, &A)) != ACP_OK) return st;
  A.px.scales = in->scales;
  A.format = in->format;
  return launched(acp::unpack8_launch(row_dtype(od.dtype), A, static_cast<hipStream_t>(stream)),
                  "unpack8 chunks " + std::to_string(A.total));
}

acp_status act_forward(acp_activation act, const acp_tile_desc* out, const acp_tile_desc* x, const acp_tile_desc* z,
                       const acp_packed8* save_x, const acp_packed8* save_z, void* stream) {
  acp::DescData od, xd, zd, cxd, czd;
  if (!known_act(act)) return ret(ACP_ERR_INVALID, "unknown activation");
  acp_status st = load_float(out, "the output", &od);
  if (st == ACP_OK) st = load_float(x, "x", &xd);
  if (st == ACP_OK && z) st = load_float(z, "z", &zd);
  if (st != ACP_OK) return st;
  const bool gated = z != nullptr, save = save_x != nullptr;
  if (save_z && !gated) return ret(ACP_ERR_INVALID, "a saved z without z");
  if (gated && (save_x != nullptr) != (save_z != nullptr))
    return ret(ACP_ERR_INVALID, "x and z are saved together or not at all");
  if (!same_shape(od, xd) || od.dtype != xd.dtype || (gated && (!same_shape(zd, xd) || zd.dtype != xd.dtype)))
    return ret(ACP_ERR_INVALID, "the operands differ in shape or dtype");
  if (save && (st = load_packed(save_x, xd, "the saved x", &cxd)) != ACP_OK) return st;
  if (save && gated) {
    if ((st = load_packed(save_z, xd, "the saved z", &czd)) != ACP_OK) return st;
    if (save_z->format != save_x->format || save_z->block != save_x->block)
      return ret(ACP_ERR_INVALID, "x and z are saved in one format and block");
  }
  if (self_overlap(od) || (save && self_overlap(cxd)) || (save && gated && self_overlap(czd)))
    return ret(ACP_ERR_INVALID, "an output overlaps itself");
  Range w[5], r[2];
  int nw = 0, nr = 0;
  w[nw++] = range_of(od, "the output");
  r[nr++] = range_of(xd, "x");
  if (gated) r[nr++] = range_of(zd, "z");
  acp::RowsArgs A{};
  const acp::DescData* t[5] = {&xd, &od};
  acp::RowTensor* rt[5] = {&A.x, &A.y};
  int nt = 2;
  if (gated) {
    t[nt] = &zd;
    rt[nt++] = &A.z;
  }
  if (save) {
    w[nw++] = range_of(cxd, "the codes of x");
    w[nw++] = range_of(save_x->scales, scale_bytes(cxd, save_x->block), "the scales of x");
    t[nt] = &cxd;
    rt[nt++] = &A.px.codes;
    A.px.scales = save_x->scales;
    A.format = save_x->format;
    if (gated) {
      w[nw++] = range_of(czd, "the codes of z");
      w[nw++] = range_of(save_z->scales, scale_bytes(czd, save_z->block), "the scales of z");
      t[nt] = &czd;
      rt[nt++] = &A.pz.codes;
      A.pz.scales = save_z->scales;
    }
  }
  if ((st = check_ranges(w, nw, r, nr)) != ACP_OK) return st;
  if (elements(xd) == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  if ((st = row_geometry(t, rt, nt, 16 / xd.esize, save ? save_x->block : 0, &A)) != ACP_OK) return st;
  A.act = act;
  return launched(acp::act_forward_launch(row_dtype(xd.dtype), gated, save, A, static_cast<hipStream_t>(stream)),
                  std::string("activation") + (gated ? " gated" : "") + (save ? " saved" : "") + " chunks " +
                      std::to_string(A.total));
}

acp_status act_backward(acp_activation act, const acp_tile_desc* dx, const acp_tile_desc* dz, const acp_tile_desc* dy,
                        const acp_packed8* x, const acp_packed8* z, void* stream) {
  acp::DescData dxd, dzd, dyd, cxd, czd;
  if (!known_act(act)) return ret(ACP_ERR_INVALID, "unknown activation");
  const bool gated = z != nullptr;
  if (gated != (dz != nullptr)) return ret(ACP_ERR_INVALID, "z and dz are given together or not at all");
  acp_status st = load_float(dy, "dy", &dyd);
  if (st == ACP_OK) st = load_float(dx, "dx", &dxd);
  if (st == ACP_OK && gated) st = load_float(dz, "dz", &dzd);
  if (st == ACP_OK) st = load_packed(x, dyd, "the saved x", &cxd);
  if (st == ACP_OK && gated) st = load_packed(z, dyd, "the saved z", &czd);
  if (st != ACP_OK) return st;
  if (!same_shape(dxd, dyd) || dxd.dtype != dyd.dtype || (gated && (!same_shape(dzd, dyd) || dzd.dtype != dyd.dtype)))
    return ret(ACP_ERR_INVALID, "the gradients differ in shape or dtype");
  if (gated && (z->format != x->format || z->block != x->block))
    return ret(ACP_ERR_INVALID, "x and z are saved in one format and block");
  if (self_overlap(dxd) || (gated && self_overlap(dzd))) return ret(ACP_ERR_INVALID, "an output overlaps itself");
  Range w[2], r[5];
  int nw = 0, nr = 0;
  acp::RowsArgs A{};
  const acp::DescData* t[5] = {&dyd, &dxd, &cxd};
  acp::RowTensor* rt[5] = {&A.dy, &A.dx, &A.px.codes};
  int nt = 3;
  w[nw++] = range_of(dxd, "dx");
  r[nr++] = range_of(dyd, "dy");
  r[nr++] = range_of(cxd, "the codes of x");
  r[nr++] = range_of(x->scales, scale_bytes(cxd, x->block), "the scales of x");
  if (gated) {
    w[nw++] = range_of(dzd, "dz");
    r[nr++] = range_of(czd, "the codes of z");
    r[nr++] = range_of(z->scales, scale_bytes(czd, z->block), "the scales of z");
    t[nt] = &dzd;
    rt[nt++] = &A.dz;
    t[nt] = &czd;
    rt[nt++] = &A.pz.codes;
    A.pz.scales = z->scales;
  }
  if ((st = check_ranges(w, nw, r, nr)) != ACP_OK) return st;
  if (elements(dyd) == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  if ((st = row_geometry(t, rt, nt, 16 / dyd.esize, x->block, &A)) != ACP_OK) return st;
  A.px.scales = x->scales;
  A.format = x->format;
  A.act = act;
  return launched(acp::act_backward_launch(row_dtype(dyd.dtype), gated, A, static_cast<hipStream_t>(stream)),
                  std::string("activation backward") + (gated ? " gated" : "") + " chunks " + std::to_string(A.total));
}

// ---------------------------------------------------------------- group norm

// The form that a norm takes (acp_dev_norm.hpp).
enum NormForm { kFormRow, kFormSlab, kFormParts };

// Workgroups that the passes over the data aim at, on 256 CUs, measured on
// [128, 500, 1024] float16 (by parts, a training step's three passes together),
// [16384, 4096] and [8192, 4096] bfloat16 (per row):
// * by parts, the pass that leaves parts: four a CU (176 us; 181 with two, 182
//   with eight, whose parts the next pass has to read), at most 256 a sample;
//   the pass that writes the result: sixteen a CU (176 us; 180 with four);
// * by parts, tensors that the eight L2s hold together: the same split for
//   both passes, a workgroup of the second where one of the first was ([4, 64,
//   64, 320] bfloat16 14.7 us with 512 workgroups in both; 16.3 with 512 and 1024,
//   21.5 with 1024 and 2048; x passes the L2s a second time all the same).
//   Few bytes take few workgroups, and so few parts ([3, 37, 41, 352] float32
//   backward 17.3 us with 256, 18.1 with 512);
// * per row: four a CU, forward (50 us; 52 with two, 61 with sixteen); backward
//   one of 512 lanes a CU (43 us; 45 with two, 50 with one of 256), since each
//   leaves 8 bytes for every channel;
// * slab, backward: a workgroup walks samples, since it leaves as much.
constexpr int64_t kNormPartial = 1024, kNormApply = 4096, kNormMaxRuns = 256;
constexpr int64_t kNormCached = 512, kNormCachedFew = 256;
constexpr int64_t kNormCachedBytes = 24 << 20, kNormFewBytes = 8 << 20;
constexpr int64_t kNormRow = 1024, kNormRowBackward = 256;
constexpr int64_t kNormSlabBackward = 1024;
// Lanes of a slab's channel block: 128 bytes of a row, a cache line
// ([128, 500, 1024] float16 66 us; 79 with 64 bytes, 71 with 256).
constexpr int64_t kSlabLanes = 8;

struct NormPlan {
  NormForm form = kFormParts;
  acp::NormArgs A{};
  acp::NormShape K{};
  acp::Div runs1{}, runs2{};  // by parts: runs of the two passes
  int64_t grid = 0;           // workgroups of its largest launch, but for the sums of columns
  int64_t workspace = 0, coef_at = 0;
  int64_t strides[4][3] = {};  // of the tensors, as RowTensor has them
  std::string text;            // acp_last_kernel's
};

// ACP_NORM_FORM=slab|parts (measurement aid): slab: not per row; parts: by
// parts whatever fits.
int norm_form_env() {
  static const int v = [] {
    const char* e = std::getenv("ACP_NORM_FORM");
    return !e ? 0 : std::strcmp(e, "slab") == 0 ? 1 : std::strcmp(e, "parts") == 0 ? 2 : 0;
  }();
  return v;
}

int64_t gcd64(int64_t a, int64_t b) { return b ? gcd64(b, a % b) : a; }
int64_t lcm64(int64_t a, int64_t b) { return a / gcd64(a, b) * b; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sizes of one norm.
struct NormDims {
  int64_t samples, rows, c, groups, per, v, block;  // block: 0 without an 8-bit form
  bool backward;
};

// About `target` runs for the steps of row_lanes rows that `rows` make, at
// least `least` steps each.
int64_t split_rows(int64_t rows, int64_t row_lanes, int64_t target, int64_t least) {
  const int64_t steps = std::max<int64_t>(1, ceil_div(rows, row_lanes));
  return std::max<int64_t>(1, std::min(target, steps / least));
}

// A row's chunks in equal channel blocks of at most 256 lanes, each a whole
// number of `unit` lanes.
void split_lanes(int64_t cpr, int64_t unit, int64_t* lanes, int64_t* blocks) {
  *blocks = ceil_div(cpr, acp::kRowThreads);
  *lanes = ceil_div(ceil_div(cpr, *blocks), unit) * unit;
  *blocks = ceil_div(cpr, *lanes);
}

void set_block(acp::NormArgs* A, int64_t lanes, int64_t blocks, int64_t threads) {
  A->lanes = div_by(static_cast<uint64_t>(lanes));
  A->blocks = div_by(static_cast<uint64_t>(blocks));
  A->row_lanes = static_cast<uint32_t>(threads / lanes);
}

// One row a sample, a group in a power of two of a wave's lanes: rows are
// samples.
bool plan_row(const NormDims& d, NormPlan* P) {
  const int64_t gl = d.per / d.v;
  if (d.rows != 1 || d.per % d.v || gl > 64 || (gl & (gl - 1))) return false;
  P->form = kFormRow;
  acp::NormArgs& A = P->A;
  int64_t lanes, blocks;
  // backward keeps no scale block together: it reads single codes
  split_lanes(d.c / d.v, std::max(gl, d.block && !d.backward ? d.block / d.v : 1), &lanes, &blocks);
  const int64_t threads = d.backward ? acp::kRowThreadsBackward : acp::kRowThreads;
  set_block(&A, lanes, blocks, threads);
  const int64_t target = (d.backward ? kNormRowBackward : kNormRow) / blocks;
  const int64_t runs = split_rows(d.samples, A.row_lanes, target, 1);
  A.runs = div_by(static_cast<uint64_t>(runs));
  A.samples = 1;
  A.rows = static_cast<uint32_t>(d.samples);
  A.group_lanes_log2 = log2_of(gl);
  P->grid = blocks * runs;
  A.main_grid = static_cast<uint32_t>(P->grid);
  A.col_rows = static_cast<uint32_t>(runs);
  P->K.threads = static_cast<uint32_t>(threads);
  P->workspace = d.backward ? runs * 2 * d.c * 4 : 0;
  return true;
}

// All rows of a sample, for a block of whole groups (and whole scale blocks
// where it saves), in a workgroup's registers.  Blocks are as narrow as leaves
// 128 bytes of a row and a chunk for each of 256 lanes, so that small tensors
// spread over many CUs.
bool plan_slab(const NormDims& d, NormPlan* P) {
  const int64_t U = d.backward ? acp::kSlabRowsBackward : acp::kSlabRows;
  // a lane's statistics are one pair, or (groups that end inside a chunk) one
  // for each channel of its chunk: those keep to 32 KiB of LDS
  const bool whole = d.per % d.v == 0;
  const int64_t most = d.backward ? acp::kSlabThreadsBackward
                                  : (whole || d.v == 4 ? acp::kSlabThreads : acp::kSlabThreads / 2);
  const bool saves = d.block && !d.backward;
  const int64_t cpr = ceil_div(d.c, d.v), align = saves ? d.block / d.v : 1;
  const int64_t unit_c = saves ? lcm64(lcm64(d.per, d.v), d.block) : lcm64(d.per, d.v);
  const int64_t unit = std::min(unit_c / d.v, ceil_div(cpr, align) * align);
  auto fits = [&](int64_t lanes, int64_t threads) { return lanes <= threads && U * (threads / lanes) >= d.rows; };
  if (!fits(unit, most)) return false;
  int64_t lanes = unit;
  while (lanes < cpr && (lanes < kSlabLanes || d.rows * lanes < 256) && fits(lanes + unit, most)) lanes += unit;
  int64_t blocks = ceil_div(cpr, lanes);
  if (blocks == 1) lanes = ceil_div(cpr, align) * align;
  if (!fits(lanes, most)) return false;
  int64_t threads = 64;
  while (!fits(lanes, threads)) threads *= 2;
  // few workgroups: more lanes with fewer chunks each
  while (threads < most && d.samples * blocks * threads <= 256 * 512 && 2 * (threads / lanes) < d.rows) threads *= 2;
  // few workgroups with long lanes, each of which waits for itself alone: by
  // parts spreads them ([1, 1024, 512] float16, 32 groups 8.8 us, 11.8 as
  // slabs of eight chunks a lane; [2, 256, 640], six, 9.2 and 8.4; [16, 1024, 512],
  // 128 workgroups, 15.4 and 13.4)
  if (!d.backward && d.samples * blocks < 64 && ceil_div(d.rows, threads / lanes) > 6) return false;
  // backward, blocks of less than 64 bytes, whose column sums take a launch of
  // their own ([8, 900, 128] float16, 8 groups 10.1 us by parts, 12.4 as slabs
  // of 32 bytes; [2, 500, 256], blocks of 64 bytes, 9.9 and 10.3)
  if (d.backward && d.samples > 1 && blocks > 1 && lanes < 4) return false;
  // backward, a lane's values fill so many registers that a CU holds one
  // workgroup of 512 lanes.  Past one a CU the form is still the fastest from
  // x itself in blocks of whole 128-byte lines ([512, 256, 1024] float16 211
  // us, by parts 230; [64, 256, 1024] 35 and 47; [1024, 200, 512] float32 250
  // and 346), but not where blocks end inside a line ([1024, 144, 320] float16
  // 126 and 99; [128, 500, 1024] in blocks of 64 bytes 132 and 117) or whose
  // codes end inside one ([512, 256, 1024] from 8 bits 63 us more)
  const bool lines = whole && !d.block && lanes % kSlabLanes == 0;
  // Samples of a few rows: by parts, each would leave as many bytes of sums as
  // it has data ([4924, 232] float16, 8 groups 66 us by parts, 27 as slabs;
  // [4000, 3, 333] bfloat16 78 and 46, but with ten rows 91 and 95; from 8 bits
  // [4000, 4, 640] forward and backward 86 and 95)
  const bool few_rows = d.rows <= (d.block ? 1 : 4);
  if (d.backward && !lines && !few_rows && d.samples * blocks * threads > 256 * 512) return false;
  // LDS that a launch may ask for without raising the kernel's limit.  Backward,
  // 16-bit rows of more than 2048 channels in one group need more and go by
  // parts, one row a sample at eight times their floor ([16384, 4096] bfloat16,
  // one group 554 us, floor 67)
  const int64_t pairs = d.backward ? threads * (d.v + 1) + lanes * d.v * 5 / 2 : threads * (whole ? 1 : d.v);
  if ((pairs + lanes * d.v / d.per + 3) * 8 > 65536) return false;
  P->form = kFormSlab;
  acp::NormArgs& A = P->A;
  set_block(&A, lanes, blocks, threads);
  const int64_t runs =
      d.backward ? std::max<int64_t>(1, std::min(d.samples, kNormSlabBackward / blocks)) : 1;
  A.runs = div_by(static_cast<uint64_t>(runs));
  A.samples = static_cast<uint32_t>(d.samples);
  A.rows = static_cast<uint32_t>(d.rows);
  P->grid = d.backward ? blocks * runs : d.samples * blocks;
  A.main_grid = static_cast<uint32_t>(P->grid);
  A.col_rows = static_cast<uint32_t>(runs);
  P->K.threads = static_cast<uint32_t>(threads);
  P->workspace = d.backward && runs > 1 ? runs * 2 * d.c * 4 : 0;
  return true;
}

bool plan_parts(const NormDims& d, NormPlan* P) {
  P->form = kFormParts;
  acp::NormArgs& A = P->A;
  int64_t lanes, blocks;
  const int64_t cpr = ceil_div(d.c, d.v);
  split_lanes(cpr, d.block && !d.backward ? d.block / d.v : 1, &lanes, &blocks);
  set_block(&A, lanes, blocks, acp::kRowThreads);
  const int64_t each = std::max<int64_t>(1, d.samples * blocks);
  const int64_t bytes = d.samples * d.rows * d.c * (16 / d.v);
  const bool cached = bytes <= kNormCachedBytes;
  const int64_t both = bytes <= kNormFewBytes ? kNormCachedFew : kNormCached;
  const int64_t first = cached ? both : kNormPartial, second = cached ? both : kNormApply;
  const int64_t runs = split_rows(d.rows, A.row_lanes, std::min(kNormMaxRuns, first / each), 2);
  P->runs1 = div_by(static_cast<uint64_t>(runs));
  const int64_t runs2 = split_rows(d.rows, A.row_lanes, second / each, 2);
  P->runs2 = div_by(static_cast<uint64_t>(runs2));
  P->grid = d.samples * blocks * std::max(runs, runs2);
  A.parts = static_cast<uint32_t>(runs);
  A.samples = static_cast<uint32_t>(d.samples);
  A.rows = static_cast<uint32_t>(d.rows);
  const int64_t width = lanes * d.v;
  A.pieces = static_cast<uint32_t>(std::min(blocks, (d.per + width - 2) / width + 1));
  A.col_rows = static_cast<uint32_t>(d.samples * runs);
  P->K.threads = acp::kRowThreads;
  const int64_t group_parts = d.samples * d.groups * runs * A.pieces * 8;
  P->coef_at = align_up(d.samples * runs * 2 * d.c * 4, 16);
  P->workspace = d.backward ? P->coef_at + group_parts : group_parts;
  return true;
}

acp_status norm_dims(const acp::DescData& t, int groups, int block, bool backward, NormDims* d) {
  const int r = t.rank;
  if (r < 2) return ret(ACP_ERR_INVALID, "group norm needs a sample dim and a channel dim");
  d->samples = t.shape[0];
  d->c = t.shape[r - 1];
  d->rows = 1;
  for (int k = 1; k + 1 < r; ++k) d->rows *= t.shape[k];
  if (d->c < 1 || d->rows < 1) return ret(ACP_ERR_INVALID, "group norm needs at least one row and one channel");
  if (groups < 1 || d->c % groups) return ret(ACP_ERR_INVALID, "the groups must divide the channels");
  if (d->samples >= kRowLimit || d->rows >= kRowLimit || d->c >= kRowLimit / 2 ||
      d->samples * ceil_div(d->c, 64) >= kRowLimit)
    return ret(ACP_ERR_UNSUPPORTED, "group norm extents go up to 2^31");
  d->groups = groups;
  d->per = d->c / groups;
  d->v = 16 / t.esize;
  d->block = block;
  d->backward = backward;
  return ACP_OK;
}

// Whether the rows of every tensor lie one stride apart, with the lanes of a
// step within the 31 bits of an offset.
bool norm_linear(const Collapsed& o, int nt, const NormDims& d, const NormPlan& P, bool by_sample,
                 const acp::DescData* const* t) {
  auto in = [&](int64_t stride) { return P.A.row_lanes * stride + 16 * P.A.lanes.d < (int64_t(1) << 31); };
  if (!by_sample && o.n > 1) return false;
  for (int k = 0; k < nt; ++k)
    if (!in(by_sample ? t[k]->strides[0] * t[k]->esize : (o.n ? o.stride[k][0] : 0))) return false;
  return !d.block || in(ceil_div(d.c, d.block) * 4);
}

// Rows of a descriptor: what a plan depends on, without its address.
struct NormKey {
  int64_t v[16 + 4 * (2 * acp::kMaxInputRank)];
  int n = 0;
  void add(int64_t x) { v[n++] = x; }
  bool operator==(const NormKey& o) const { return n == o.n && std::memcmp(v, o.v, sizeof(int64_t) * n) == 0; }
};

std::string norm_text(const NormDims& d, const NormPlan& P) {
  static const char* const forms[] = {" per row", " slab", " by parts"};
  static const char* const kinds[] = {" whole", " split", " any"};
  return std::string(d.backward ? "group norm backward" : "group norm") +
         (d.block ? (d.backward ? " from 8 bits" : " saved") : "") + forms[P.form] + kinds[P.K.kind] + " threads " +
         std::to_string(P.K.threads) + " lanes " + std::to_string(P.A.lanes.d) + "x" + std::to_string(P.A.row_lanes) +
         " blocks " + std::to_string(P.A.blocks.d) + " runs " +
         std::to_string(P.form == kFormParts ? P.runs1.d : P.A.runs.d) +
         (P.form == kFormParts ? "+" + std::to_string(P.runs2.d) : std::string());
}

// The first form that holds.  `row_linear` and `slab_linear` say of such a plan
// whether the tensors' strides allow it.
template <class R, class S>
NormPlan choose_form(const NormDims& d, R row_linear, S slab_linear) {
  const int env = norm_form_env();
  NormPlan row, slab, parts;
  if (env < 1 && plan_row(d, &row) && row_linear(row)) return row;
  if (env < 2 && plan_slab(d, &slab) && slab_linear(slab)) return slab;
  plan_parts(d, &parts);
  return parts;
}

// The form, split and strides of a norm over `t` (of one shape).
acp_status norm_geometry(const acp::DescData* const* t, int nt, const NormDims& d, NormPlan* out) {
  Collapsed o;
  if (!collapse(t, nt, 1, 2, &o))
    return ret(ACP_ERR_UNSUPPORTED, "the inner row dims of these strides do not join into two");
  NormPlan P = choose_form(d, [&](const NormPlan& p) { return norm_linear(o, nt, d, p, true, t); },
                           [&](const NormPlan& p) { return norm_linear(o, nt, d, p, false, t); });
  const bool row = P.form == kFormRow;
  acp::NormArgs& A = P.A;
  const bool linear = P.form != kFormParts || norm_linear(o, nt, d, P, false, t);
  P.K.kind = !linear || d.c % d.v ? acp::kNormAny : d.per % d.v ? acp::kNormSplit : acp::kNormWhole;
  P.K.dt = row_dtype(t[0]->dtype);
  A.c = static_cast<uint32_t>(d.c);
  A.groups = static_cast<uint32_t>(d.groups);
  A.per_group = static_cast<uint32_t>(d.per);
  A.per = div_by(static_cast<uint64_t>(d.per));
  A.lb_log2 = d.block ? log2_of(d.block / d.v) : 0;
  A.row2 = div_by(static_cast<uint64_t>(row ? std::max<int64_t>(1, d.samples) : (o.n >= 1 ? o.ext[o.n - 1] : 1)));
  const int64_t scale_row = d.block ? ceil_div(d.c, d.block) * 4 : 0;
  A.scales.s[0] = row ? 0 : scale_row * d.rows;
  A.scales.s[1] = row ? 0 : scale_row * A.row2.d;
  A.scales.s[2] = scale_row;
  for (int k = 0; k < nt; ++k) {
    const int64_t sample = t[k]->strides[0] * t[k]->esize;
    P.strides[k][0] = row ? 0 : sample;
    P.strides[k][1] = !row && o.n >= 2 ? o.stride[k][0] : 0;
    P.strides[k][2] = row ? sample : (o.n >= 1 ? o.stride[k][o.n - 1] : 0);
  }
  // a launch has fewer than 2^32 lanes; backward by parts the columns are in
  // the second pass's, else in one of their own
  const int64_t columns = d.backward ? ceil_div(2 * d.c, acp::kColumns) : 0;
  const int64_t wg = P.form == kFormParts ? P.grid + columns : P.grid;
  if (std::max(wg * int64_t(P.K.threads), columns * acp::kRowThreads) >= int64_t(1) << 32)
    return ret(ACP_ERR_UNSUPPORTED, "a launch of 2^32 lanes");
  P.text = norm_text(d, P);
  *out = P;
  return ACP_OK;
}

// The plan of a norm over `t`, with the tensors' addresses in their places.
// Each thread keeps the plans of its last few geometries (shapes, strides and
// types; no addresses): planning costs as much as a launch.
acp_status norm_plan(const acp::DescData* const* t, int nt, const NormDims& d, NormPlan* out) {
  NormKey key;
  for (int64_t x : {int64_t(t[0]->dtype), int64_t(t[0]->rank), d.groups, d.block, int64_t(d.backward), int64_t(nt)})
    key.add(x);
  for (int k = 0; k < t[0]->rank; ++k) key.add(t[0]->shape[k]);
  for (int k = 0; k < nt; ++k) {
    key.add(t[k]->esize);
    for (int e = 0; e < t[k]->rank; ++e) key.add(t[k]->strides[e]);
  }
  struct Entry {
    NormKey key;
    NormPlan plan;
  };
  constexpr int kEntries = 16;
  thread_local Entry entries[kEntries];
  thread_local int next = 0;
  for (const Entry& e : entries)
    if (e.key == key) {
      *out = e.plan;
      return ACP_OK;
    }
  const acp_status st = norm_geometry(t, nt, d, out);
  if (st != ACP_OK) return st;
  Entry& e = entries[next];
  next = (next + 1) % kEntries;
  e.key = key;
  e.plan = *out;
  return ACP_OK;
}

void set_tensor(const NormPlan& P, int k, const acp::DescData& d, acp::RowTensor* t) {
  t->p = reinterpret_cast<char*>(d.gbase);
  for (int e = 0; e < 3; ++e) t->s[e] = P.strides[k][e];
}

bool misaligned4(const void* p) { return reinterpret_cast<uint64_t>(p) % 4 != 0; }

acp_status check_workspace(const void* workspace, int64_t bytes, int64_t need, int64_t samples) {
  if (need == 0 || samples == 0) return ACP_OK;
  if (!workspace || bytes < need)
    return ret(ACP_ERR_INVALID, "the workspace is smaller than acp_group_norm_workspace says");
  if (reinterpret_cast<uint64_t>(workspace) % 16) return ret(ACP_ERR_INVALID, "the workspace is not 16-byte aligned");
  return ACP_OK;
}

acp_status group_norm_workspace(const acp_tile_desc* x, int groups, int64_t* bytes) {
  acp::DescData xd;
  if (!bytes) return ret(ACP_ERR_INVALID, "null argument");
  const acp_status st = load_float(x, "x", &xd);
  if (st != ACP_OK) return st;
  // The most of the forms that calls take: the other tensors' strides may turn
  // a norm per row into a slab, and a slab of several rows into parts; a form is
  // never asked for that no call takes (by parts, samples of one row would leave
  // two to four times their own bytes)
  NormDims d;
  const acp_status sd = norm_dims(xd, groups, 0, false, &d);
  if (sd != ACP_OK) return sd;
  int64_t need = 0;
  auto calls = [&](bool row_linear, bool slab_linear) {
    for (bool backward : {false, true})
      for (int block : {0, 32, 64, 128, 256}) {
        d.backward = backward;
        d.block = block;
        need = std::max(need, choose_form(d, [&](const NormPlan&) { return row_linear; },
                                          [&](const NormPlan&) { return slab_linear; }).workspace);
      }
  };
  calls(true, true);
  calls(false, true);
  if (d.rows > 1) calls(false, false);
  *bytes = need;
  return ret(ACP_OK);
}

acp_status group_norm(const acp_tile_desc* y, const acp_tile_desc* x, const float* gamma, const float* beta,
                      int groups, float eps, acp_activation act, float* mean, float* rstd, const acp_packed8* save,
                      void* workspace, int64_t workspace_bytes, void* stream) {
  acp::DescData xd, yd, cd;
  acp_status st = load_float(x, "x", &xd);
  if (st == ACP_OK) st = load_float(y, "y", &yd);
  if (st != ACP_OK) return st;
  if (!known_act(act)) return ret(ACP_ERR_INVALID, "unknown activation");
  if (!(eps >= 0.0f) || std::isinf(eps)) return ret(ACP_ERR_INVALID, "eps must be a finite number >= 0");
  if (!same_shape(xd, yd) || xd.dtype != yd.dtype) return ret(ACP_ERR_INVALID, "x and y differ in shape or dtype");
  if (save && (st = load_packed(save, xd, "the saved x", &cd)) != ACP_OK) return st;
  if (misaligned4(gamma) || misaligned4(beta) || misaligned4(mean) || misaligned4(rstd))
    return ret(ACP_ERR_INVALID, "a float32 array is not 4-byte aligned");
  NormDims d;
  if ((st = norm_dims(xd, groups, save ? save->block : 0, false, &d)) != ACP_OK) return st;
  NormPlan P;
  acp::NormArgs& A = P.A;
  const acp::DescData* t[] = {&xd, &yd, &cd};
  if ((st = norm_plan(t, save ? 3 : 2, d, &P)) != ACP_OK) return st;
  set_tensor(P, 0, xd, &A.x);
  set_tensor(P, 1, yd, &A.y);
  if (save) {
    set_tensor(P, 2, cd, &A.codes);
    A.scales.p = reinterpret_cast<char*>(save->scales);
  }
  if ((st = check_workspace(workspace, workspace_bytes, P.workspace, d.samples)) != ACP_OK) return st;
  if (self_overlap(yd) || (save && self_overlap(cd))) return ret(ACP_ERR_INVALID, "an output overlaps itself");
  const int64_t stat = d.samples * groups * 4;
  Range w[6] = {range_of(yd, "y"), range_of(mean, stat, "mean"), range_of(rstd, stat, "rstd"),
                range_of(workspace, P.workspace, "the workspace")};
  int nw = 4;
  if (save) {
    w[nw++] = range_of(cd, "the codes");
    w[nw++] = range_of(save->scales, scale_bytes(cd, save->block), "the scales");
  }
  const Range r[] = {range_of(xd, "x"), range_of(gamma, d.c * 4, "gamma"), range_of(beta, d.c * 4, "beta")};
  if ((st = check_ranges(w, nw, r, 3)) != ACP_OK) return st;
  if (elements(xd) == 0) return launched_nothing();
  if ((st = check_stream(stream)) != ACP_OK) return st;
  P.K.packed = save ? 1 + save->format : 0;
  P.K.act = act;
  A.gamma = gamma;
  A.beta = beta;
  A.mean = mean;
  A.rstd = rstd;
  A.part = static_cast<float*>(workspace);
  A.eps = eps;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (P.form == kFormRow) e = acp::norm_launch(acp::kNormOpRow, P.K, A, s);
  if (P.form == kFormSlab) e = acp::norm_launch(acp::kNormOpSlab, P.K, A, s);
  if (P.form == kFormParts) {
    A.runs = P.runs1;
    A.main_grid = A.samples * A.blocks.d * A.runs.d;
    e = acp::norm_launch(acp::kNormOpStats, P.K, A, s);
    A.runs = P.runs2;
    A.main_grid = A.samples * A.blocks.d * A.runs.d;
    if (e == hipSuccess) e = acp::norm_launch(acp::kNormOpApply, P.K, A, s);
  }
  return launched(e, P.text);
}

acp_status group_norm_backward(const acp_tile_desc* dx, float* dgamma, float* dbeta, const acp_tile_desc* dy,
                               const acp_tile_desc* x, const acp_packed8* saved, const float* mean, const float* rstd,
                               const float* gamma, const float* beta, int groups, acp_activation act, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  acp::DescData dxd, dyd, xd, cd;
  if ((x != nullptr) == (saved != nullptr)) return ret(ACP_ERR_INVALID, "give x or its saved form, and not both");
  acp_status st = load_float(dy, "dy", &dyd);
  if (st == ACP_OK) st = load_float(dx, "dx", &dxd);
  if (st == ACP_OK && x) st = load_float(x, "x", &xd);
  if (st == ACP_OK && saved) st = load_packed(saved, dyd, "the saved x", &cd);
  if (st != ACP_OK) return st;
  if (!known_act(act)) return ret(ACP_ERR_INVALID, "unknown activation");
  if (!mean || !rstd) return ret(ACP_ERR_INVALID, "the backward pass needs mean and rstd");
  if (!same_shape(dxd, dyd) || dxd.dtype != dyd.dtype || (x && (!same_shape(xd, dyd) || xd.dtype != dyd.dtype)))
    return ret(ACP_ERR_INVALID, "x, dy and dx differ in shape or dtype");
  if (misaligned4(gamma) || misaligned4(beta) || misaligned4(mean) || misaligned4(rstd) || misaligned4(dgamma) ||
      misaligned4(dbeta))
    return ret(ACP_ERR_INVALID, "a float32 array is not 4-byte aligned");
  NormDims d;
  if ((st = norm_dims(dyd, groups, saved ? saved->block : 0, true, &d)) != ACP_OK) return st;
  NormPlan P;
  acp::NormArgs& A = P.A;
  const acp::DescData* t[] = {&dyd, &dxd, x ? &xd : &cd};
  if ((st = norm_plan(t, 3, d, &P)) != ACP_OK) return st;
  set_tensor(P, 0, dyd, &A.dy);
  set_tensor(P, 1, dxd, &A.dx);
  set_tensor(P, 2, *t[2], x ? &A.x : &A.codes);
  if (saved) A.scales.p = reinterpret_cast<char*>(saved->scales);
  if ((st = check_workspace(workspace, workspace_bytes, P.workspace, d.samples)) != ACP_OK) return st;
  if (self_overlap(dxd)) return ret(ACP_ERR_INVALID, "an output overlaps itself");
  const int64_t stat = d.samples * groups * 4;
  const Range w[] = {range_of(dxd, "dx"), range_of(dgamma, d.c * 4, "dgamma"), range_of(dbeta, d.c * 4, "dbeta"),
                     range_of(workspace, P.workspace, "the workspace")};
  Range r[7] = {range_of(dyd, "dy"), range_of(mean, stat, "mean"), range_of(rstd, stat, "rstd"),
                range_of(gamma, d.c * 4, "gamma"), range_of(beta, d.c * 4, "beta")};
  int nr = 5;
  if (x) r[nr++] = range_of(xd, "x");
  if (saved) {
    r[nr++] = range_of(cd, "the codes");
    r[nr++] = range_of(saved->scales, scale_bytes(cd, saved->block), "the scales");
  }
  if ((st = check_ranges(w, 4, r, nr)) != ACP_OK) return st;
  P.K.packed = saved ? 1 + saved->format : 0;
  P.K.act = act;
  A.gamma = gamma;
  A.beta = beta;
  A.mean = const_cast<float*>(mean);
  A.rstd = const_cast<float*>(rstd);
  A.dgamma = dgamma;
  A.dbeta = dbeta;
  A.part = static_cast<float*>(workspace);
  A.coef = reinterpret_cast<float*>(static_cast<char*>(workspace) + P.coef_at);
  if ((st = check_stream(stream)) != ACP_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (elements(dyd) == 0) {  // no samples: the gradients of the parameters are zero
    A.col_rows = 0;
    if (!dgamma && !dbeta) return launched_nothing();
    return launched(acp::norm_columns_launch(A, s), "group norm backward of no samples");
  }
  if (P.form == kFormRow) e = acp::norm_launch(acp::kNormOpRowBackward, P.K, A, s);
  if (P.form == kFormSlab) e = acp::norm_launch(acp::kNormOpSlabBackward, P.K, A, s);
  if (P.form == kFormParts) {
    A.runs = P.runs1;
    A.main_grid = A.samples * A.blocks.d * A.runs.d;
    e = acp::norm_launch(acp::kNormOpSums, P.K, A, s);
    A.runs = P.runs2;
    A.main_grid = A.samples * A.blocks.d * A.runs.d;
    if (e == hipSuccess) e = acp::norm_launch(acp::kNormOpDx, P.K, A, s);
  } else if (P.workspace > 0 && e == hipSuccess) {
    e = acp::norm_columns_launch(A, s);
  }
  return launched(e, P.text);
}

// Nothing throws across the ABI.
template <class F>
acp_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return ACP_ERR_INVALID;
  }
}

}  // namespace

extern "C" {

acp_status acp_pack8(const acp_packed8* out, const acp_tile_desc* x, void* hip_stream) {
  return guarded([&] { return pack8(out, x, hip_stream); });
}

acp_status acp_unpack8(const acp_tile_desc* out, const acp_packed8* in, void* hip_stream) {
  return guarded([&] { return unpack8(out, in, hip_stream); });
}

acp_status acp_act_forward(acp_activation act, const acp_tile_desc* out, const acp_tile_desc* x,
                           const acp_tile_desc* z, const acp_packed8* save_x, const acp_packed8* save_z,
                           void* hip_stream) {
  return guarded([&] { return act_forward(act, out, x, z, save_x, save_z, hip_stream); });
}

acp_status acp_act_backward(acp_activation act, const acp_tile_desc* dx, const acp_tile_desc* dz,
                            const acp_tile_desc* dy, const acp_packed8* x, const acp_packed8* z, void* hip_stream) {
  return guarded([&] { return act_backward(act, dx, dz, dy, x, z, hip_stream); });
}

acp_status acp_group_norm_workspace(const acp_tile_desc* x, int groups, int64_t* bytes) {
  return guarded([&] { return group_norm_workspace(x, groups, bytes); });
}

acp_status acp_group_norm(const acp_tile_desc* y, const acp_tile_desc* x, const float* gamma, const float* beta,
                          int groups, float eps, acp_activation act, float* mean, float* rstd,
                          const acp_packed8* save, void* workspace, int64_t workspace_bytes, void* hip_stream) {
  return guarded([&] {
    return group_norm(y, x, gamma, beta, groups, eps, act, mean, rstd, save, workspace, workspace_bytes, hip_stream);
  });
}

acp_status acp_group_norm_backward(const acp_tile_desc* dx, float* dgamma, float* dbeta, const acp_tile_desc* dy,
                                   const acp_tile_desc* x, const acp_packed8* saved, const float* mean,
                                   const float* rstd, const float* gamma, const float* beta, int groups,
                                   acp_activation act, void* workspace, int64_t workspace_bytes, void* hip_stream) {
  return guarded([&] {
    return group_norm_backward(dx, dgamma, dbeta, dy, x, saved, mean, rstd, gamma, beta, groups, act, workspace,
                               workspace_bytes, hip_stream);
  });
}

}  // extern "C"
