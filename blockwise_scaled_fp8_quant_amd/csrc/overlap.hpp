// Whether tensors that a call writes share memory with others that it reads or writes, for the argument checks of
// abi_ops.cpp.  Tensors are rows in memory: columns of one buffer side by side are apart, however their spans interleave.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <utility>

namespace puro {

// `groups` times `rows` rows of `width` bytes: row r of group g begins at lo + g * ld_group + r * ld_row.
struct Rows {
  typedef __int128 wide;      // (strides are the caller's numbers: products may pass 64 bits)
  wide lo;
  int64_t groups, rows;
  wide ld_group, ld_row, width;
  bool replaces = false;      // may be the very rows of another such tensor: an output in its input's place

  wide hi() const { return lo + (groups - 1) * ld_group + (rows - 1) * ld_row + width; }
};

inline Rows matrix(const void* p, int64_t n, int64_t ld, int64_t columns, int64_t es) {
  return Rows{(Rows::wide) reinterpret_cast<uintptr_t>(p), n, 1, (Rows::wide)ld * es, 0, (Rows::wide)columns * es};
}
inline Rows replacing(Rows r) {
  r.replaces = true;
  return r;
}
inline Rows vector(const void* p, uintptr_t bytes) {
  return Rows{(Rows::wide) reinterpret_cast<uintptr_t>(p), 1, 1, 0, 0, (Rows::wide)bytes};
}

// v / d towards minus infinity, held within [0, n - 1]
inline int64_t step_below(Rows::wide v, Rows::wide d, int64_t n) {
  if (n <= 1 || v <= 0 || d <= 0) return 0;
  const Rows::wide q = v / d;
  return q > n - 1 ? n - 1 : (int64_t)q;
}

// Whether [lo, hi) meets a row of b, whose rows and groups lie apart and in order.
inline bool meets(const Rows& b, Rows::wide lo, Rows::wide hi) {
  // of the rows that end behind lo the first one decides: it is the last that begins at or before lo, or the next
  const auto row = [&](int64_t g, int64_t r) {
    const Rows::wide at = b.lo + g * b.ld_group + r * b.ld_row;
    return at < hi && at + b.width > lo;
  };
  const int64_t g = step_below(lo - b.lo, b.ld_group, b.groups);
  const int64_t r = step_below(lo - b.lo - g * b.ld_group, b.ld_row, b.rows);
  return row(g, r) || (r + 1 < b.rows && row(g, r + 1)) || (g + 1 < b.groups && row(g + 1, 0));
}

inline bool same_strides(const Rows& a, const Rows& b) {
  return a.groups == b.groups && a.rows == b.rows && a.width == b.width && (a.groups == 1 || a.ld_group == b.ld_group) &&
         (a.rows == 1 || a.ld_row == b.ld_row);
}

// Whether a (any strides from 0 on) and b (rows and groups apart and in order) share memory.
inline bool share_memory(Rows a, const Rows& b) {
  if (a.lo >= b.hi() || b.lo >= a.hi()) return false;
  if (same_strides(a, b)) {
    // the same strides: rows (g, r) and (g', r') meet where the distance of the tensors, some strides on, is below a row; a row's
    // place in its group is less than a group's stride, so that two differences of the groups are left, and two of the rows
    const Rows::wide distance = a.lo - b.lo;
    const auto nearest = [](Rows::wide v, Rows::wide ld, int64_t n, int64_t k) -> Rows::wide {      // -v / ld, k = 0 below, 1 above
      if (n == 1) return 0;
      const Rows::wide q = -v / ld;
      const Rows::wide below = q * ld > -v ? q - 1 : q;
      const Rows::wide at = below + k;
      return at < 1 - (Rows::wide)n ? 1 - (Rows::wide)n : at > n - 1 ? n - 1 : at;
    };
    for (int64_t i = 0; i < 2; ++i) {
      const Rows::wide left = distance + nearest(distance, b.ld_group, b.groups, i) * b.ld_group;
      for (int64_t k = 0; k < 2; ++k) {
        const Rows::wide d = left + nearest(left, b.ld_row, b.rows, k) * b.ld_row;
        if (d < b.width && -d < b.width) return true;
      }
    }
    return false;
  }
  // rows of a that adjoin or repeat are one
  if (a.ld_row > a.ld_group && a.groups > 1) {
    std::swap(a.ld_row, a.ld_group);
    std::swap(a.rows, a.groups);
  }
  if (a.rows > 1 && a.ld_row <= a.width) {
    a.width += (a.rows - 1) * a.ld_row;
    a.rows = 1;
  }
  if (a.groups > 1 && a.rows == 1 && a.ld_group <= a.width) {
    a.width += (a.groups - 1) * a.ld_group;
    a.groups = 1;
  }
  for (int64_t g = 0; g < a.groups; ++g)
    for (int64_t r = 0; r < a.rows; ++r) {
      const Rows::wide at = a.lo + g * a.ld_group + r * a.ld_row;
      if (meets(b, at, at + a.width)) return true;
    }
  return false;
}

// The tensors of a call.  Each that is written has its rows apart.
class Tensors {
 public:
  void reads(const void* p, const Rows& r) {
    if (p && r.width > 0) in_[n_in_++] = Spanned{r, r.hi()};
  }
  void writes(const void* p, const Rows& r) {
    if (p && r.width > 0) out_[n_out_++] = Spanned{r, r.hi()};
  }
  // Whether one that is written shares memory with another that it does not replace.
  bool clash() const {
    for (int i = 0; i < n_out_; ++i) {
      for (int k = 0; k < n_in_; ++k)
        if (meet(in_[k], out_[i]) && !replaced(in_[k].rows, out_[i].rows) && share_memory(in_[k].rows, out_[i].rows)) return true;
      for (int k = 0; k < i; ++k)
        if (meet(out_[k], out_[i]) && share_memory(out_[k].rows, out_[i].rows)) return true;
    }
    return false;
  }

 private:
  struct Spanned {
    Rows rows;
    Rows::wide end;
  };
  // (the spans of nearly all pairs are apart)
  static bool meet(const Spanned& a, const Spanned& b) { return a.rows.lo < b.end && b.rows.lo < a.end; }
  static bool replaced(const Rows& in, const Rows& out) {
    return in.replaces && out.replaces && in.lo == out.lo && same_strides(in, out);
  }
  Spanned in_[12], out_[12];
  int n_in_ = 0, n_out_ = 0;
};

}  // namespace puro
