// Shared parts of the dense FP4 operators: the matrix's layout, rows of 16 or 32
// bits, and the host checks of both.
#pragma once

#include "common.cuh"
#include "fp4.h"
#include "fp4_span.h"

namespace fp4 {

constexpr int kMaxCols = 32768, kMaxRows = 1 << 24;

__host__ __device__ __forceinline__ int block_of(int format) { return format == MOE_FMT_NVFP4 ? 16 : 32; }
// Tiles of 4 scales that a row has.
__host__ __device__ __forceinline__ int scale_tiles(int cols, int format) {
  const int span = 4 * block_of(format);
  return (cols + span - 1) / span;
}
// Byte of the first of the 4 scales that row r has in tile kt.
__device__ __forceinline__ size_t scale_word(int r, int kt, int tiles) {
  return ((size_t)(r >> 7) * tiles + kt) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

// Rows of 16 or 32 bits, as the entry points' arguments describe them.
struct Rows {
  void* data;
  long long stride;
  int type;
};
inline Rows rows_of(const void* data, long long stride, int type) { return Rows{const_cast<void*>(data), stride, type}; }

// ---------------------------------------------------------------------------
// Host checks
// ---------------------------------------------------------------------------

inline bool shape_ok(int rows, int cols, int format) {
  return rows >= 0 && rows <= kMaxRows && cols >= 32 && cols <= kMaxCols && cols % 32 == 0 &&
         (format == MOE_FMT_NVFP4 || format == MOE_FMT_MXFP4);
}

inline int check_matrix(const fp4_matrix* m) {
  if (!m || m->rows < 0) return MOE_ERR_INVALID_ARG;
  if (!shape_ok(m->rows, m->cols, m->format)) return MOE_ERR_UNSUPPORTED;
  if (m->rows > 0 && (!m->codes || !m->scales)) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(m->codes) || !moe::aligned16(m->scales) || ((uintptr_t)m->row_scale & 3u))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}
// ... that is written.
inline int check_target(const fp4_matrix* m, int rows, int cols) {
  if (const int rc = check_matrix(m)) return rc;
  if (m->rows != rows || m->cols != cols) return MOE_ERR_INVALID_ARG;
  if (m->format == MOE_FMT_NVFP4 && rows > 0 && !m->row_scale) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

__host__ __device__ __forceinline__ int element_bytes(int type) { return type == FP4_FP32 ? 4 : 2; }

// Rows that are read or written 16 bytes at a time.  `wide`: 32-bit rows are allowed.
inline int check_rows(const Rows& x, int rows, int cols, bool wide) {
  if (!x.data && rows > 0) return MOE_ERR_INVALID_ARG;
  if (x.type != FP4_BF16 && x.type != FP4_FP16 && !(wide && x.type == FP4_FP32)) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned16(x.data)) return MOE_ERR_ALIGNMENT;
  if (rows > 1 && (x.stride < cols || x.stride >= (1ll << 38))) return MOE_ERR_INVALID_ARG;
  if (rows > 1 && x.stride % (16 / element_bytes(x.type)) != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Where operands lie.  `elements`: rows that their kernel reads and writes element by element.
inline Span span_of(const Rows& x, int rows, int cols, bool elements) {
  Span s = rows_span(x.data, rows, cols, x.stride, element_bytes(x.type));
  if (!elements) s.item = 0;
  return s;
}
inline Span codes_span(const fp4_matrix& m) { return piece(m.codes, (long long)m.rows * m.cols / 2); }
inline Span scales_span(const fp4_matrix& m) {
  return piece(m.scales, (long long)((m.rows + 127) / 128) * scale_tiles(m.cols, m.format) * 512);
}
inline Span row_scale_span(const fp4_matrix& m) { return piece(m.row_scale, (long long)m.rows * 4); }

}  // namespace fp4
