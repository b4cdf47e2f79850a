// Four neighbouring bf16 by each lane of a warp, 128 columns of a row, where the
// row begins at any element: the warp reads the aligned 8-byte pieces that hold
// them, and lanes pass the parts on.
#pragma once

#include <cuda_bf16.h>

namespace xp {

// How many elements before a column that is a multiple of 4 its piece begins.
__device__ __forceinline__ int ahead_of(const __nv_bfloat16* row) { return (int)(reinterpret_cast<unsigned long long>(row) >> 1) & 3; }

// Whether a row's first and last pieces lie within the matrix, of which `before`
// elements are before the row and `behind` from its beginning on.
__device__ __forceinline__ bool pieces_inside(unsigned long long before, unsigned long long behind, unsigned cols) { return before >= 3 && behind >= cols + 3ull; }

// The piece from element e of a row of `cols` (none: zeros): with what lies
// before and behind the row, but where that is not the matrix's.
__device__ __forceinline__ uint2 piece_at(const __nv_bfloat16* row, int e, int cols, bool inside) {
  uint2 q = make_uint2(0, 0);
  if (cols <= max(e, 0)) return q;
  if (inside || (e >= 0 && e + 4 <= cols)) {
    q = *reinterpret_cast<const uint2*>(row + e);
  } else {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(row);
    unsigned long long v = 0;
#pragma unroll 1
    for (int i = 3; i >= 0; --i) v = v << 16 | (e + i >= 0 && e + i < cols ? h[e + i] : 0u);
    q = make_uint2((unsigned)v, (unsigned)(v >> 32));
  }
  return q;
}

// Columns c .. c + 3 of a lane, zeros behind the row, from its piece q and the
// next lane's.  The last lane's next piece is `more` of lane `from`.  The whole
// warp calls it.
__device__ __forceinline__ uint2 join_pieces(uint2 q, uint2 more, int from, int s, unsigned c, unsigned cols) {
  if (s) {
    const int lane = threadIdx.x & 31;
    unsigned nx = __shfl_sync(0xffffffffu, q.x, (lane + 1) & 31), ny = __shfl_sync(0xffffffffu, q.y, (lane + 1) & 31);
    const unsigned mx = __shfl_sync(0xffffffffu, more.x, from), my = __shfl_sync(0xffffffffu, more.y, from);
    if (lane == 31) nx = mx, ny = my;
    const unsigned a = s & 2 ? q.y : q.x, b = s & 2 ? nx : q.y, d = s & 2 ? ny : nx;
    q = make_uint2(__funnelshift_r(a, b, 16 * (s & 1)), __funnelshift_r(b, d, 16 * (s & 1)));
  }
  const int n = (int)cols - (int)c;
  if (n < 4) q = make_uint2(n < 1 ? 0u : n < 2 ? q.x & 0xffffu : q.x, n < 3 ? 0u : q.y & 0xffffu);
  return q;
}

}  // namespace xp
