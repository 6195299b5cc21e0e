// norm_rows.h -- which bytes layer normalisation reads of a row by 16-byte
// vectors.  A row of d elements may start and end within a vector.  Plain
// integer arithmetic, so that a test can run it on the host.
#pragma once

#ifdef __CUDACC__
#define GDR_ROWS_FN __host__ __device__ __forceinline__
#else
#define GDR_ROWS_FN inline
#endif

namespace gdr {
namespace rows {

// Where a row whose first element is number `at` of its tensor starts within
// its first vector of V elements, and how many vectors it touches.
GDR_ROWS_FN int shift(long long at, int V) { return (int)(at & (V - 1)); }
GDR_ROWS_FN int vectors(int shift, int d, int V) {
  return (shift + d + V - 1) / V;
}

// Whether the tensor can end within a vector of a row of token `tok`: its last
// one holds up to V - 1 elements of what follows, and every later token has at
// least one.
GDR_ROWS_FN bool may_end(long long tok, int ntok, int V) {
  return tok > ntok - V;
}
// Bytes to read then, with `left` elements of `es` bytes from the vector's
// start to the tensor's end.
GDR_ROWS_FN int vector_bytes(long long left, int V, int es) {
  return left < V ? (int)left * es : V * es;
}

}  // namespace rows
}  // namespace gdr
