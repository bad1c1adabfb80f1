// Checks of the block operators' arguments: token rows with strides, vectors
// per batch element, and whether two tensors share memory.
#pragma once

#include <cstdint>

namespace flux {

// Rows [B, S] of `width` elements of `size` bytes, strides in elements.
struct Rows {
  const void *p;
  int64_t B, S, width, bs, rs;
  int size;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Largest extent in elements of one tensor (a tensor map's strides stay below
// 2^40 bytes).
constexpr int64_t kMaxSpan = int64_t{1} << 38;

// Strides that no size looks at get those of contiguous rows.
inline void settle(Rows &t) {
  if (t.S == 1) t.rs = (t.width + 7) / 8 * 8;
  if (t.B == 1) t.bs = t.rs <= kMaxSpan / t.S ? t.S * t.rs : t.rs;
}

// Strides are multiples of 8 elements, no smaller than a row, and the rows fit
// the span.
inline bool strides_ok(const Rows &t) {
  if (t.rs <= 0 || t.bs <= 0 || t.rs % 8 != 0 || t.bs % 8 != 0) return false;
  if (t.rs > kMaxSpan / t.S || t.bs > kMaxSpan / t.B) return false;
  return (t.S == 1 || t.rs >= t.width) && (t.B == 1 || t.bs >= t.width);
}

// No two rows of the tensor share an element (an output's condition): batch
// elements follow one another, or interleave between the tokens of the first.
inline bool rows_disjoint(const Rows &t) {
  if (t.S > 1 && t.rs < t.width) return false;
  if (t.B > 1 && t.bs < t.width) return false;
  if (t.S == 1 || t.B == 1) return true;
  return t.bs >= (t.S - 1) * t.rs + t.width || t.rs >= (t.B - 1) * t.bs + t.width;
}

inline int64_t span_bytes(const Rows &t) {
  return ((t.B - 1) * t.bs + (t.S - 1) * t.rs + t.width) * t.size;
}

inline bool ranges_meet(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(nb) && b0 < a0 + static_cast<uintptr_t>(na);
}

// Whether two tensors share a byte. Tensors with the same strides (views of
// one buffer: two streams of a joint sequence, two blocks of its columns) are
// decided row by row; others by the address ranges they span.
inline bool share(const Rows &a, const Rows &b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  if (!ranges_meet(a.p, span_bytes(a), b.p, span_bytes(b))) return false;
  if (a.bs * a.size != b.bs * b.size && a.B > 1 && b.B > 1) return true;
  if (a.rs * a.size != b.rs * b.size && a.S > 1 && b.S > 1) return true;
  // row (i, j) of b starts `off` + i * big + j * small bytes after row (i', j')
  // of a, differences i - i' and j - j' within the sizes
  struct Axis {
    int64_t step, lo, hi;
  };
  Axis big{(a.B > 1 ? a.bs * a.size : b.bs * b.size), -(a.B - 1), b.B - 1};
  Axis small{(a.S > 1 ? a.rs * a.size : b.rs * b.size), -(a.S - 1), b.S - 1};
  if (big.step < small.step) {
    const Axis t = big;
    big = small;
    small = t;
  }
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p)) -
                      static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p));
  const int64_t wa = a.width * a.size, wb = b.width * b.size;
  // rows meet when -wb < distance < wa; the long axis leaves few candidates
  const int64_t reach = (small.hi > -small.lo ? small.hi : -small.lo) * small.step + wa + wb;
  int64_t i0 = (-off - reach) / big.step - 1, i1 = (-off + reach) / big.step + 1;
  if (i0 < big.lo) i0 = big.lo;
  if (i1 > big.hi) i1 = big.hi;
  if (i1 - i0 > 4096) return true;
  for (int64_t i = i0; i <= i1; ++i) {
    const int64_t d = off + i * big.step;
    int64_t j0 = (-wb - d) / small.step - 1, j1 = (wa - d) / small.step + 1;
    if (j0 < small.lo) j0 = small.lo;
    if (j1 > small.hi) j1 = small.hi;
    for (int64_t j = j0; j <= j1; ++j) {
      const int64_t e = d + j * small.step;
      if (e > -wb && e < wa) return true;
    }
  }
  return false;
}

// A vector per batch element (gate, scale, shift): [B, width] at stride bs,
// which may be 0 (one vector for all).
inline bool vec_stride_ok(int64_t bs, int64_t B) {
  return bs >= 0 && bs % 8 == 0 && bs <= kMaxSpan / B;
}
inline Rows vec_rows(const void *p, int64_t B, int64_t width, int64_t bs, int f32) {
  if (bs == 0 || B == 1) return Rows{p, 1, 1, width, width, width, f32 ? 4 : 2};
  return Rows{p, B, 1, width, bs, width, f32 ? 4 : 2};
}

constexpr int64_t kMaxTokens = int64_t{1} << 30;

// Batch elements that follow one another at the token stride are one run of
// tokens.
inline bool joins(const Rows &t) { return t.p == nullptr || t.B == 1 || t.bs == t.S * t.rs; }

}  // namespace flux
