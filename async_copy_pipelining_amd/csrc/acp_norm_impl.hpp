// Group norm for one element type: picks the kernel of a pass and launches it.
// Included by one translation unit a type.
#pragma once

#include "acp_dev_norm_bwd.hpp"
#include "acp_dev_norm_fwd.hpp"

namespace acp {
namespace norm {

template <int I>
using Int = std::integral_constant<int, I>;

// A kernel's arguments out of a call's.
inline void pick(const NormArgs& a, NormStats* u) {
  static_cast<NormCore&>(*u) = a;
  u->x = a.x;
}
inline void pick(const NormArgs& a, NormForward* u) {
  static_cast<NormCore&>(*u) = a;
  u->x = a.x;
  u->y = a.y;
}
inline void pick(const NormArgs& a, NormForwardSaved* u) {
  pick(a, static_cast<NormForward*>(u));
  u->codes = a.codes;
  u->scales = a.scales;
}
inline void pick(const NormArgs& a, NormBackward* u) {
  static_cast<NormCore&>(*u) = a;
  u->dy = a.dy;
  u->dx = a.dx;
  u->x = a.x;
}
inline void pick(const NormArgs& a, NormBackwardSaved* u) {
  static_cast<NormCore&>(*u) = a;
  u->dy = a.dy;
  u->dx = a.dx;
  u->codes = a.codes;
  u->scales = a.scales;
}

template <class A>
hipError_t launch(void (*kernel)(A), const NormArgs& a, uint32_t grid, uint32_t threads, uint32_t lds, hipStream_t s) {
  std::remove_const_t<A> u;
  pick(a, &u);
  void* args[] = {&u};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(threads), args, lds, s);
}

// f(kind), f(packed, act) and so on with the shape's values as types
template <class F>
hipError_t by_kind(const NormShape& k, F f) {
  return k.kind == kNormWhole ? f(Int<kNormWhole>()) : k.kind == kNormSplit ? f(Int<kNormSplit>()) : f(Int<kNormAny>());
}
template <class F>
hipError_t by_form(const NormShape& k, F f) {
  auto with_act = [&](auto pk) {
    return k.act == dev::kActSilu ? f(pk, Int<dev::kActSilu>())
                                  : k.act == dev::kActGelu ? f(pk, Int<dev::kActGelu>()) : f(pk, Int<dev::kActNone>());
  };
  return k.packed == 0 ? with_act(Int<0>()) : k.packed == 1 ? with_act(Int<1>()) : with_act(Int<2>());
}

// groups that one channel block may touch
inline uint32_t block_groups(const NormArgs& a, int v) {
  const uint32_t g = (a.lanes.d * static_cast<uint32_t>(v) - 1) / a.per_group + 2;
  return g < a.groups ? g : a.groups;
}

// LDS of channel_sums, and `n` pairs and a float for each channel of a block
inline uint32_t sums_lds(const NormArgs& a, int v, uint32_t threads, uint32_t n) {
  return threads * static_cast<uint32_t>(v + 1) * 8u + a.lanes.d * static_cast<uint32_t>(v) * (n * 8u + 4u);
}

template <class T>
hipError_t run(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s) {
  constexpr int V = dev::kChunk<T>;
  switch (op) {
    case kNormOpRow:
      return by_form(k, [&](auto pk, auto act) {
        return launch(dev::norm_row_kernel<T, pk(), act()>, a, a.main_grid, kRowThreads, 0, s);
      });
    case kNormOpSlab: {
      const uint32_t lds = (k.threads * (k.kind == kNormWhole ? 1 : V) + block_groups(a, V)) * 8u;
      return by_kind(k, [&](auto kind) {
        return by_form(k, [&](auto pk, auto act) {
          return launch(dev::norm_slab_kernel<T, kind(), pk(), act()>, a, a.main_grid, k.threads, lds, s);
        });
      });
    }
    case kNormOpStats:
      return by_kind(k, [&](auto kind) {
        return launch(dev::norm_stats_kernel<T, kind()>, a, a.main_grid, kRowThreads, 0, s);
      });
    case kNormOpApply:
      return by_kind(k, [&](auto kind) {
        return by_form(k, [&](auto pk, auto act) {
          return launch(dev::norm_apply_kernel<T, kind(), pk(), act()>, a, a.main_grid, kRowThreads,
                        block_groups(a, V) * 8u, s);
        });
      });
    case kNormOpRowBackward:
      return by_form(k, [&](auto pk, auto act) {
        return launch(dev::norm_row_backward_kernel<T, pk(), act()>, a, a.main_grid, k.threads,
                      sums_lds(a, V, k.threads, 1), s);
      });
    case kNormOpSlabBackward: {
      const uint32_t width = a.lanes.d * static_cast<uint32_t>(V);
      const uint32_t lds = sums_lds(a, V, k.threads, 2) + (width / a.per_group + 1) * 8u;
      return by_kind(k, [&](auto kind) {
        return by_form(k, [&](auto pk, auto act) {
          return launch(dev::norm_slab_backward_kernel<T, kind(), pk(), act()>, a, a.main_grid, k.threads, lds, s);
        });
      });
    }
    case kNormOpSums:
      return by_kind(k, [&](auto kind) {
        return by_form(k, [&](auto pk, auto act) {
          return launch(dev::norm_sums_kernel<T, kind(), pk(), act()>, a, a.main_grid, kRowThreads,
                        sums_lds(a, V, kRowThreads, 1), s);
        });
      });
    case kNormOpDx:
      return by_kind(k, [&](auto kind) {
        return by_form(k, [&](auto pk, auto act) {
          return launch(dev::norm_dx_kernel<T, kind(), pk(), act()>, a, a.main_grid + norm_column_grid(a), kRowThreads,
                        block_groups(a, V) * 8u, s);
        });
      });
  }
  return hipErrorInvalidValue;
}

}  // namespace norm
}  // namespace acp
