// Where an operand of a dense FP4 operator lies, and whether two of them share bytes.
// Operands may be strided views of one buffer (gate | up | out side by side in a row), so
// that their ranges meet while their rows do not: rows are compared, not ranges.
// Host only, plain C++.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace fp4 {

// `rows` rows of `width` bytes, `stride` >= width bytes apart.  `item`: bytes of an element where a
// kernel writes only what the same thread has read before, if both lie at the same place; else 0.
struct Span {
  long long at, width, stride, rows;
  int item;
};
// n bytes in one piece; nothing where there is no address.
inline Span piece(const void* p, long long n) { return Span{(long long)(uintptr_t)p, n, n, p && n > 0 ? 1 : 0, 0}; }
inline Span rows_span(const void* p, long long rows, long long cols, long long stride, int item) {
  if (!p || rows <= 0) return piece(nullptr, 0);
  if (rows == 1 || stride <= 0) return Span{(long long)(uintptr_t)p, cols * item, cols * item, 1, item};
  return Span{(long long)(uintptr_t)p, cols * item, stride * item, rows, item};
}

inline bool same_place(const Span& a, const Span& b) {
  return a.item && a.item == b.item && a.at == b.at && a.width == b.width && a.stride == b.stride && a.rows == b.rows;
}

// Whether bytes p .. p + n - 1 meet a row: the first row that does not end before them starts before their end.
inline bool meets(long long p, long long n, const Span& s) {
  const long long past = p - s.at - s.width;  // the row at `at + r * stride` ends behind p if r * stride > past
  const long long r = past < 0 ? 0 : past / s.stride + 1;
  return r < s.rows && s.at + r * s.stride < p + n;
}

inline bool overlap(Span a, Span b) {
  if (!a.rows || !b.rows) return false;
  auto end = [](const Span& s) { return s.at + (s.rows - 1) * s.stride + s.width; };
  if (end(a) <= b.at || end(b) <= a.at) return false;
  for (Span* s : {&a, &b})
    if (s->width == s->stride) s->width *= s->rows, s->stride = s->width, s->rows = 1;
  if (a.rows == 1) return meets(a.at, a.width, b);
  if (b.rows == 1) return meets(b.at, b.width, a);
  if (a.stride == b.stride) {
    // All rows of b that have rows of a on both sides lie alike between them.  Row j of b starts in the
    // stride of row q + j of a: the first that meets one is the one before row 0's stride, or the next.
    const long long d = b.at - a.at, q = d >= 0 ? d / a.stride : -((-d + a.stride - 1) / a.stride);
    const long long j = q < 0 ? -q - 1 : 0;
    return (j < b.rows && meets(b.at + j * b.stride, b.width, a)) ||
           (j + 1 < b.rows && meets(b.at + (j + 1) * b.stride, b.width, a));
  }
  // (of unequal strides, in one buffer: no ordinary layout; some ns a row)
  const Span &few = a.rows < b.rows ? a : b, &many = a.rows < b.rows ? b : a;
  for (long long r = 0; r < few.rows; ++r)
    if (meets(few.at + r * few.stride, few.width, many)) return true;
  return false;
}

// Whether no output shares bytes with an input or with another output, but for those at the
// same place as an input that is read element by element.
template <int N, int M>
inline bool apart(const Span (&outs)[N], const Span (&ins)[M]) {
  for (int i = 0; i < N; ++i) {
    for (int k = 0; k < M; ++k)
      if (!same_place(outs[i], ins[k]) && overlap(outs[i], ins[k])) return false;
    for (int k = 0; k < i; ++k)
      if (overlap(outs[i], outs[k])) return false;
  }
  return true;
}

}  // namespace fp4
