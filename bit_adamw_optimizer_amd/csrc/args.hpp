// args.hpp -- argument checks that the C ABI's files share (train_abi.hip,
// model_abi.hip): types, shapes, the memory of a call's arguments. Internal.
#pragma once

#include <stdint.h>

#include <string>

#include "host.hpp"
#include "msamp.h"

namespace msamp {

// Elements of a matrix's address range: keeps every offset, in bytes too,
// within 63 bits.
constexpr int64_t kMaxSpan = (int64_t)1 << 58;
constexpr int64_t kMaxCols = INT32_MAX;

inline msamp_status invalid(const std::string& msg) { return fail(MSAMP_E_INVALID_ARG, msg); }

inline int64_t elem_size(int dtype) { return dtype == MSAMP_F32 ? 4 : 2; }

inline msamp_status check_dtype(int dtype, const char* role) {
  if (dtype != MSAMP_F32 && dtype != MSAMP_F16 && dtype != MSAMP_BF16)
    return invalid(std::string("unknown ") + role);
  return MSAMP_OK;
}

inline msamp_status check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return invalid("a size is negative");
  if (cols > kMaxCols) return invalid("cols exceeds 2^31 - 1");
  if (rows > kMaxSpan) return invalid("rows exceeds 2^58");
  return MSAMP_OK;
}

// A matrix of rows x cols elements of 'size' bytes; not NULL unless empty.
inline msamp_status check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size, bool written,
                          const char* role) {
  if (rows == 0 || cols == 0) return MSAMP_OK;
  if (p == nullptr) return invalid(std::string(role) + " is NULL");
  if (((uintptr_t)p & (uintptr_t)(size - 1)) != 0)
    return fail(MSAMP_E_MISALIGNED, std::string(role) + " is not aligned to its elements");
  if (ld < 0 || (written && rows > 1 && ld < cols))
    return invalid(std::string(role) + ": the distance between rows is " + (ld < 0 ? "negative" : "less than a row"));
  if (ld > 0 && rows - 1 > (kMaxSpan - cols) / ld) return invalid(std::string(role) + " spans too much memory");
  return MSAMP_OK;
}

inline msamp_status check_vector(const void* p, int64_t n, int64_t size, const char* role) {
  return check_matrix(p, 1, n, n, size, true, role);
}

inline msamp_status check_checkpoint(const msamp_checkpoint* c, int64_t rows, int64_t cols, bool written, const char* role) {
  if (c == nullptr) return invalid(std::string(role) + " is NULL");
  if (c->fmt != MSAMP_FP8_E4M3 && c->fmt != MSAMP_FP8_E5M2)
    return invalid(std::string(role) + ": unknown FP8 format");
  MSAMP_TRY(check_matrix(c->codes, rows, cols, c->ld, 1, written, (std::string(role) + ".codes").c_str()));
  const int64_t groups = (cols + MSAMP_CHECKPOINT_GROUP - 1) / MSAMP_CHECKPOINT_GROUP;
  return check_matrix(c->scales, rows, groups, c->ld_scales, 1, written, (std::string(role) + ".scales").c_str());
}

// The memory of a call's arguments. What is written may share none with
// anything else (the kernels write some rows while they still read others),
// but some outputs may be an input: equal matrices of the same number other
// than 0 in 'in_place', of which one is written, each element of it by the
// lanes that have read it.
class Regions {
 public:
  void add(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size, bool written, const char* role,
           int in_place = 0, int64_t outer = 0) {
    if (p == nullptr || rows == 0 || cols == 0) return;
    r_[n_++] = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)(((rows - 1) * ld + cols) * size), cols * size,
                rows == 1 ? cols * size : ld * size, outer, rows == 1, written, in_place, role, {}};
  }
  // [batch, time, cols] with distances sb and st: the rows of a matrix where
  // one distance is a multiple of the other (with the rows between them, which
  // may be nobody's), otherwise all that lies between the first and the last.
  // Two of the same distances, one of them beyond all that the other spans, are
  // compared row by row (rows_meet).
  void cube(const void* p, int64_t batch, int64_t time, int64_t cols, int64_t sb, int64_t st, int64_t size,
            bool written, const char* role, int in_place) {
    if (p == nullptr || batch == 0 || time == 0 || cols == 0) return;
    if (batch == 1) sb = 0;
    if (time == 1) st = 0;
    const int64_t small = batch == 1 ? st : time == 1 ? sb : st < sb ? st : sb, large = st < sb ? sb : st;
    const int64_t last = (batch - 1) * sb + (time - 1) * st;  // the last row's start
    if (batch == 1 && time == 1) add(p, 1, cols, cols, size, written, role, in_place, 0);
    else if (small >= cols && (small == large || batch == 1 || time == 1 || large % small == 0))
      add(p, last / small + 1, cols, small, size, written, role, in_place, sb);
    else add(p, 1, last + cols, last + cols, size, written, role, in_place, sb);
    const int64_t n = small == st ? time : batch;  // rows 'small' apart
    if (batch > 1 && time > 1 && small >= cols && large >= (n - 1) * small + cols)
      r_[n_ - 1].rows = {cols * size, small * size, large * size, n, batch * time / n};
  }
  void vector(const void* p, int64_t n, int64_t size, bool written, const char* role) {
    add(p, 1, n, n, size, written, role);
  }
  void checkpoint(const msamp_checkpoint* c, int64_t rows, int64_t cols, bool written, const char* role) {
    if (c == nullptr) return;
    add(c->codes, rows, cols, c->ld, 1, written, role);
    add(c->scales, rows, (cols + MSAMP_CHECKPOINT_GROUP - 1) / MSAMP_CHECKPOINT_GROUP, c->ld_scales, 1, written, role);
  }
  msamp_status check() const {
    for (int i = 1; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((r_[i].written || r_[j].written) && overlap(r_[i], r_[j]))
          return invalid(std::string(r_[j].role) + " and " + r_[i].role + " overlap");
    return MSAMP_OK;
  }

 private:
  struct Rows {  // of a cube, in bytes: runs of 'count' rows 'small' apart, 'large' apart; bytes 0: not such a cube
    int64_t bytes, small, large, count, runs;
  };
  struct Region {
    uintptr_t lo, hi;
    int64_t row, ld, outer;
    bool one, written;
    int in_place;
    const char* role;
    Rows rows;
  };
  // Whether a row of one cube touches a row of another of the same distances:
  // rows i runs and j rows apart do where the starts' distance less i large and
  // j small is less than a row, which only the nearest two i and j can make it.
  static bool rows_meet(const Region& a, const Region& b) {
    const Rows& r = a.rows;
    const int64_t d = (int64_t)(b.lo - a.lo);
    auto below = [](int64_t v, int64_t by) { return v / by - (v % by < 0 ? 1 : 0); };
    const int64_t i0 = below(d, r.large);
    for (int64_t i = i0; i <= i0 + 1; ++i) {
      const int64_t left = d - i * r.large, j0 = below(left, r.small);
      for (int64_t j = j0; j <= j0 + 1; ++j) {
        const int64_t apart = left - j * r.small;
        if (i > -r.runs && i < r.runs && j > -r.count && j < r.count && apart > -r.bytes && apart < r.bytes) return true;
      }
    }
    return false;
  }
  static bool overlap(const Region& a, const Region& b) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    if (a.in_place != 0 && a.in_place == b.in_place && !(a.written && b.written) && a.lo == b.lo && a.hi == b.hi &&
        a.row == b.row && a.outer == b.outer && (a.ld == b.ld || a.one))
      return false;
    if (a.rows.bytes != 0 && a.rows.bytes == b.rows.bytes && a.rows.small == b.rows.small &&
        a.rows.large == b.rows.large && a.rows.count == b.rows.count && a.rows.runs == b.rows.runs)
      return rows_meet(a, b);
    // rows side by side at the same distance (columns of one buffer)
    const int64_t ld = a.one ? b.ld : a.ld;
    if ((a.one && b.one) || (!a.one && !b.one && a.ld != b.ld) || ld == 0) return true;
    const int64_t d = b.lo >= a.lo ? (int64_t)((b.lo - a.lo) % (uintptr_t)ld)
                                   : (ld - (int64_t)((a.lo - b.lo) % (uintptr_t)ld)) % ld;
    return d < a.row || d + b.row > ld;
  }
  Region r_[16];
  int n_ = 0;
};

// [batch, time, cols]: a matrix of each sequence. One that is written has no
// element twice.
inline msamp_status check_cube(const void* p, int64_t batch, int64_t time, int64_t cols, int64_t sb, int64_t st,
                               int64_t size, bool written, const char* role) {
  if (batch == 0 || time == 0 || cols == 0) return MSAMP_OK;
  MSAMP_TRY(check_matrix(p, time, cols, st, size, written, role));
  MSAMP_TRY(check_matrix(p, batch, cols, sb, size, written, role));
  if (time == 1) st = 0;
  if (batch == 1) sb = 0;
  if ((batch - 1) * sb > kMaxSpan - cols - (time - 1) * st) return invalid(std::string(role) + " spans too much memory");
  if (written && batch > 1 && time > 1 && sb < (time - 1) * st + cols && st < (batch - 1) * sb + cols)
    return invalid(std::string(role) + ": its sequences overlap");
  return MSAMP_OK;
}

inline msamp_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return MSAMP_OK;
  if (ws == nullptr) return invalid("workspace is NULL");
  if (((uintptr_t)ws & 15u) != 0) return fail(MSAMP_E_MISALIGNED, "workspace is not 16-byte aligned");
  if (bytes < need)
    return invalid("workspace has " + std::to_string(bytes) + " bytes, " + std::to_string(need) + " are needed");
  return MSAMP_OK;
}

template <typename F>
int64_t workspace_of(F&& f) {
  int64_t bytes = -1;
  guarded([&]() -> msamp_status {
    clear_error();
    return f(&bytes);
  });
  return bytes;
}

}  // namespace msamp
