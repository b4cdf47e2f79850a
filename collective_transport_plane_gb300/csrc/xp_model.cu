// Host side of include/xp_model.h: argument checks, the products' tiles and
// tensor maps, and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "xp_checks.h"
#include "xp_model_internal.h"
#include "xp_train_internal.h"

namespace {

using namespace xp::checks;

bool is_block_rows(int n) { return n == 1 || n == XP_BLOCK8; }
int shift_of(int block_rows) { return block_rows == 1 ? 0 : 7; }
size_t ceil_div(size_t a, size_t b) { return (a + b - 1) / b; }

xp_status check_shape(size_t rows, size_t cols) {
  if (rows > XP_MODEL_MAX_ROWS) return fail(XP_ERR_INVALID, "rows %zu above 2^28", rows);
  if (cols > XP_MODEL_MAX_COLS) return fail(XP_ERR_INVALID, "cols %zu above 2^20", cols);
  return XP_OK;
}
xp_status check_types(int dtype, int wdtype) {
  if (!is_float_type(dtype) || !is_float_type(wdtype)) return fail(XP_ERR_INVALID, "dtype %d / %d is neither XP_F32 nor XP_BF16", dtype, wdtype);
  return XP_OK;
}
xp_status check_matrix(const char* what, const void* p, size_t stride, size_t rows, size_t cols, int dtype) {
  if (stride > XP_MODEL_MAX_STRIDE) return fail(XP_ERR_INVALID, "%s: rows %zu elements apart", what, stride);
  return check_rows(what, p, stride, rows, cols, dtype);
}
// Whether every row begins at a multiple of `a` bytes.
bool rows_aligned(const void* p, size_t stride, size_t rows, size_t es, size_t a) { return aligned(p, a) && (rows == 1 || stride * es % a == 0); }

// Codes and scales of a matrix in 8 bits.
xp_status check_block8(const char* what, const uint8_t* codes, size_t stride, const uint8_t* scales, size_t scales_stride, size_t rows,
                       size_t cols, int block_rows) {
  char name[64];
  snprintf(name, sizeof name, "%s's scales", what);
  xp_status s = check_matrix(what, codes, stride, rows, cols, XP_U8);
  if (s != XP_OK) return s;
  return check_matrix(name, scales, scales_stride, ceil_div(rows, block_rows), ceil_div(cols, XP_BLOCK8), XP_U8);
}
Span span8(const uint8_t* p, size_t stride, size_t rows, size_t cols) { return span_of(p, stride, rows, cols, 1); }
Span span_scales(const uint8_t* p, size_t stride, size_t rows, size_t cols, int block_rows) {
  return span_of(p, stride, ceil_div(rows, block_rows), ceil_div(cols, XP_BLOCK8), 1);
}

// The first of `written` that shares bytes with another of them or with one of `read`.
template <size_t W, size_t R>
bool any_overlap(const Span (&written)[W], size_t nw, const Span (&read)[R], size_t nr) {
  for (size_t i = 0; i < nw; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return true;
    for (size_t j = 0; j < nr; ++j)
      if (overlap(written[i], read[j])) return true;
  }
  return false;
}

int sm_count() {
  static xp::PerDevice known;
  return known.get([](int dev) {
    int n = 0;
    return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0 ? n : 1;
  });
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess || found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}
// Whether a matrix's blocks of 128 codes are lines of L2.
bool on_lines(const uint8_t* codes, size_t stride, size_t rows) { return rows_aligned(codes, stride, rows, 1, 128); }

// Boxes of 128 codes by box_rows rows, swizzled over 128 bytes, zeros outside the matrix.  What L2 fetches is widened to
// 256 bytes where a row's blocks are lines of it, and left alone where they straddle lines (4096 x 5120 x 16001, rows
// 16016 bytes apart: 325 us with it, 288 without; 16000 x 16000 by one row, rows 16000 bytes apart: 47 and 48).
bool map_codes(CUtensorMap* map, const uint8_t* codes, size_t stride, size_t rows, size_t cols, unsigned box_rows) {
  const cuuint64_t size[2] = {cols, rows}, pitch[1] = {rows == 1 ? round_up(cols, 16) : stride};
  const cuuint32_t box[2] = {XP_BLOCK8, box_rows}, step[2] = {1, 1};
  return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), size, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, on_lines(codes, stride, rows) ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product is cut: tiles of 128 of b's rows (256 for a pair of CTAs) and bn
// of a's, and the CTAs that share one.  The least of a model in ns, fitted to
// times of all choices at 27 sizes (N = K = 4096: 64 rows 9.1 us as 4 CTAs a tile,
// 12.5 as one, 10.2 in pairs; 512 rows 12.8 in pairs of 128, 14.8 alone; 4096 rows
// 42 in pairs of 224, 46 of 256, which have room in TMEM for one tile's sums
// only, 52 alone): a block's copies and products, which take longer where blocks
// straddle L2's lines, what a tile's last sums take, and what CTAs that share a
// tile add.  Into how many parts the columns are cut decides the order of the
// additions, so it is chosen as if rows lay on lines, wherever they lie: equal
// products give equal bits in any layout.  (Choices for rows off lines by themselves
// had other parts at 2% of sizes: 192 x 2048 x 4096 11.0 us, 9.8 so; 2024 x 435 x
// 11067 21.9 and 19.3; 620 x 3028 x 12890 27.7 and 29.4.)
void cut_product(size_t m, size_t n, size_t kblocks, unsigned sms, bool lines, xp::Matmul8Params& p) {
  static const unsigned widths[] = {16, 32, 64, 96, 128, 160, 192, 224, 256};
  struct Cut {
    size_t cost;
    unsigned ctas, bn;
  } cuts[4] = {{~(size_t)0, 0, 0}, {~(size_t)0, 0, 0}, {~(size_t)0, 0, 0}, {~(size_t)0, 0, 0}};   // the least for 1, 2, 4 and 8 parts
  size_t least = ~(size_t)0;
  unsigned parts = 0;   // a power of 2
  for (unsigned ctas = 1; ctas <= 2; ++ctas) {
    const unsigned whole = (unsigned)std::min<size_t>(256, round_up(m, 16 * ctas));
    const size_t tiles_p = ceil_div(n, 128 * ctas), units = std::max(1u, sms / ctas);
    for (unsigned width : widths) {
      const unsigned bn = std::min(width, whole);
      if (bn % (16 * ctas)) continue;
      const size_t tiles = tiles_p * ceil_div(m, bn), waves = ceil_div(tiles, units);
      const size_t on = ctas == 1 ? 150u + bn * 23 / 20 : std::max(150u, 120u + bn);
      const size_t off = ctas == 1 ? on + bn * 9 / 10 : std::max(150u, 120u + bn * 5 / 4);
      for (unsigned i = 0; i < (ctas == 2 ? 1u : 4u); ++i) {
        const unsigned split = 1u << i;
        // (clusters of 8 find room for 64 CTAs: with 128 they came one after another)
        if (split > 1 && (split > kblocks || tiles * split > (split == 8 ? std::min(64u, sms) : sms))) break;
        const auto cost = [&](size_t block) {
          return waves * (ceil_div(kblocks, split) * block + (bn > 224 ? 1000 : 0)) + 5500 + 4 * bn + (split > 1 ? 1200 + 11 * bn : 0);
        };
        if (cost(on) < least) least = cost(on), parts = i;
        const size_t here = cost(lines ? on : off);
        if (here < cuts[i].cost) cuts[i] = {here, ctas, bn};
      }
      if (bn == whole) break;
    }
  }
  p.ctas = cuts[parts].ctas;
  p.bn = cuts[parts].bn;
  p.split = 1u << parts;
  p.tiles_p = (unsigned)ceil_div(n, 128 * p.ctas);
  p.tiles_q = (unsigned)ceil_div(m, p.bn);
}

// A backward pass's workspace, whatever its type and alignment: long rows' sums, and rows of partial sums.
size_t rms_workspace(size_t rows, size_t cols, int sms) {
  size_t most = 0;
  for (int dtype : {XP_F32, XP_BF16})
    for (bool wide : {false, true}) {
      const xp::RmsBackwardShape s = xp::rms_backward_shape(rows, cols, dtype, wide, sms);
      most = std::max(most, (s.is_long ? round_up(rows * 4, 16) : 0) + s.nparts * cols * sizeof(float));
    }
  return most;
}

xp_status check_distill(const void* logits, size_t stride, const int32_t* ids, const float* teacher, size_t rows, size_t vocab, size_t top,
                        float temperature, int dtype) {
  xp_status s = check_shape(rows, vocab);
  if (s != XP_OK || (s = check_types(dtype, dtype)) != XP_OK) return s;
  if (vocab == 0) return fail(XP_ERR_INVALID, "vocab is 0");
  if (top > XP_DISTILL_MAX_TOP) return fail(XP_ERR_INVALID, "top %zu above 1024", top);
  // 1e-6 to 1e6: its square and its inverse times any logit of use stay within fp32
  if (!(temperature >= 1e-6f && temperature <= 1e6f)) return fail(XP_ERR_INVALID, "temperature %g not in [1e-6, 1e6]", temperature);
  if (rows == 0) return XP_OK;
  if (top && (!ids || !teacher || !aligned(ids, 4) || !aligned(teacher, 4))) return fail(XP_ERR_INVALID, "ids or teacher is NULL or not aligned to its element");
  return check_matrix("logits", logits, stride, rows, vocab, dtype);
}

}  // namespace

extern "C" {

xp_status xp_block8_encode(const void* x, size_t x_stride, size_t rows, size_t cols, xp_dtype dtype, int block_rows, uint8_t* codes,
                           size_t codes_stride, uint8_t* scales, size_t scales_stride, uint8_t* codes_t, size_t codes_t_stride,
                           uint8_t* scales_t, size_t scales_t_stride, xp_stream_t stream) {
  xp_status s = check_shape(rows, cols);
  if (s != XP_OK || (s = check_types(dtype, dtype)) != XP_OK) return s;
  if (!is_block_rows(block_rows)) return fail(XP_ERR_INVALID, "block_rows %d is neither 1 nor 128", block_rows);
  if (!codes && !codes_t) return fail(XP_ERR_INVALID, "codes and codes_t are NULL");
  if (codes_t && rows > XP_MODEL_MAX_COLS) return fail(XP_ERR_INVALID, "rows %zu above 2^20, the columns of a transposed matrix", rows);
  if (rows == 0 || cols == 0) return XP_OK;
  if ((s = check_matrix("x", x, x_stride, rows, cols, dtype)) != XP_OK) return s;
  if (codes && (s = check_block8("codes", codes, codes_stride, scales, scales_stride, rows, cols, block_rows)) != XP_OK) return s;
  if (codes_t && (s = check_block8("codes_t", codes_t, codes_t_stride, scales_t, scales_t_stride, cols, rows, block_rows)) != XP_OK) return s;
  const size_t es = size_of(dtype);
  const Span read[1] = {span_of(x, x_stride, rows, cols, es)};
  Span written[4];
  size_t n = 0;
  if (codes) written[n++] = span8(codes, codes_stride, rows, cols), written[n++] = span_scales(scales, scales_stride, rows, cols, block_rows);
  if (codes_t) written[n++] = span8(codes_t, codes_t_stride, cols, rows), written[n++] = span_scales(scales_t, scales_t_stride, cols, rows, block_rows);
  if (any_overlap(written, n, read, 1)) return fail(XP_ERR_INVALID, "x, codes and scales overlap");
  const size_t tiles_c = ceil_div(cols, 128);
  if (tiles_c * ceil_div(rows, 128) > 0x7fffffff) return fail(XP_ERR_INVALID, "%zu x %zu elements are too many", rows, cols);
  xp::Encode8Params p = {};
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.codes_t = codes_t;
  p.scales_t = scales_t;
  p.x_stride = x_stride;
  p.codes_stride = codes_stride;
  p.scales_stride = scales_stride;
  p.codes_t_stride = codes_t_stride;
  p.scales_t_stride = scales_t_stride;
  p.rows = (unsigned)rows;
  p.cols = (unsigned)cols;
  p.tiles_c = (unsigned)tiles_c;
  p.tiles = (unsigned)(tiles_c * ceil_div(rows, 128));
  p.x_aligned = rows_aligned(x, x_stride, rows, es, 4 * es);
  p.codes_aligned = rows_aligned(codes, codes_stride, rows, 1, 4);
  p.codes_t_aligned = rows_aligned(codes_t, codes_t_stride, cols, 1, 4);
  p.all_aligned = p.x_aligned && (!codes || p.codes_aligned) && (!codes_t || p.codes_t_aligned);
  XP_CUDA(xp::launch_encode8(p, dtype, block_rows, sm_count(), stream));
  return XP_OK;
}

xp_status xp_block8_decode(const uint8_t* codes, size_t codes_stride, const uint8_t* scales, size_t scales_stride, size_t rows, size_t cols,
                           int block_rows, void* out, size_t out_stride, xp_dtype dtype, xp_stream_t stream) {
  xp_status s = check_shape(rows, cols);
  if (s != XP_OK || (s = check_types(dtype, dtype)) != XP_OK) return s;
  if (!is_block_rows(block_rows)) return fail(XP_ERR_INVALID, "block_rows %d is neither 1 nor 128", block_rows);
  if (rows == 0 || cols == 0) return XP_OK;
  if ((s = check_block8("codes", codes, codes_stride, scales, scales_stride, rows, cols, block_rows)) != XP_OK) return s;
  if ((s = check_matrix("out", out, out_stride, rows, cols, dtype)) != XP_OK) return s;
  const size_t es = size_of(dtype);
  const Span read[2] = {span8(codes, codes_stride, rows, cols), span_scales(scales, scales_stride, rows, cols, block_rows)};
  const Span written[1] = {span_of(out, out_stride, rows, cols, es)};
  if (any_overlap(written, 1, read, 2)) return fail(XP_ERR_INVALID, "codes, scales and out overlap");
  if (ceil_div(ceil_div(cols, 256) * rows, 8) > 0x7fffffff) return fail(XP_ERR_INVALID, "%zu x %zu elements are too many", rows, cols);
  xp::Decode8Params p = {};
  p.codes = codes;
  p.scales = scales;
  p.out = out;
  p.codes_stride = codes_stride;
  p.scales_stride = scales_stride;
  p.out_stride = out_stride;
  p.rows = (unsigned)rows;
  p.cols = (unsigned)cols;
  p.shift = shift_of(block_rows);
  p.aligned = rows_aligned(codes, codes_stride, rows, 1, 8) && rows_aligned(out, out_stride, rows, es, 16);
  XP_CUDA(xp::launch_decode8(p, dtype, stream));
  return XP_OK;
}

xp_status xp_matmul8(const uint8_t* a, size_t a_stride, const uint8_t* a_scales, size_t a_scales_stride, int a_block_rows, const uint8_t* b,
                     size_t b_stride, const uint8_t* b_scales, size_t b_scales_stride, int b_block_rows, void* c, size_t c_stride, size_t m,
                     size_t n, size_t k, xp_dtype c_dtype, int accumulate, xp_stream_t stream) {
  xp_status s = check_shape(m, k);
  if (s != XP_OK || (s = check_shape(n, k)) != XP_OK || (s = check_types(c_dtype, c_dtype)) != XP_OK) return s;
  if (!is_block_rows(a_block_rows) || !is_block_rows(b_block_rows))
    return fail(XP_ERR_INVALID, "block_rows %d / %d is neither 1 nor 128", a_block_rows, b_block_rows);
  if (accumulate && c_dtype != XP_F32) return fail(XP_ERR_INVALID, "only an fp32 c is added to");
  if (m == 0 || n == 0) return XP_OK;
  if ((s = check_matrix("c", c, c_stride, m, n, c_dtype)) != XP_OK) return s;
  const size_t es = size_of(c_dtype);
  if (k == 0) {
    if (!accumulate) XP_CUDA(cudaMemset2DAsync(c, (m == 1 ? n : c_stride) * es, 0, n * es, m, stream));
    return XP_OK;
  }
  if ((s = check_block8("a", a, a_stride, a_scales, a_scales_stride, m, k, a_block_rows)) != XP_OK) return s;
  if ((s = check_block8("b", b, b_stride, b_scales, b_scales_stride, n, k, b_block_rows)) != XP_OK) return s;
  if (!rows_aligned(a, a_stride, m, 1, 16) || !rows_aligned(b, b_stride, n, 1, 16))
    return fail(XP_ERR_INVALID, "rows of a or b do not begin at multiples of 16 bytes");
  if (!rows_aligned(a_scales, a_scales_stride, ceil_div(m, a_block_rows), 1, 4) || !rows_aligned(b_scales, b_scales_stride, ceil_div(n, b_block_rows), 1, 4))
    return fail(XP_ERR_INVALID, "rows of scales do not begin at multiples of 4 bytes");
  const Span read[4] = {span8(a, a_stride, m, k), span_scales(a_scales, a_scales_stride, m, k, a_block_rows), span8(b, b_stride, n, k),
                        span_scales(b_scales, b_scales_stride, n, k, b_block_rows)};
  const Span written[1] = {span_of(c, c_stride, m, n, es)};
  if (any_overlap(written, 1, read, 4)) return fail(XP_ERR_INVALID, "c overlaps a, b or their scales");
  if (!encode_tiled()) return fail(XP_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  xp::Matmul8Params p = {};
  const size_t kblocks = ceil_div(k, XP_BLOCK8);
  const int sms = sm_count();
  cut_product(m, n, kblocks, (unsigned)sms, on_lines(a, a_stride, m) && on_lines(b, b_stride, n), p);
  if ((size_t)p.tiles_p * p.tiles_q > 0x7fffffff) return fail(XP_ERR_INVALID, "%zu x %zu elements are too many", m, n);
  if (!map_codes(&p.p_map, b, b_stride, n, k, 128) || !map_codes(&p.q_map, a, a_stride, m, k, p.bn / p.ctas))
    return fail(XP_ERR_CUDA, "cuTensorMapEncodeTiled refuses %zu x %zu or %zu x %zu codes", m, k, n, k);
  p.p_scales = b_scales;
  p.q_scales = a_scales;
  p.p_pitch = b_scales_stride;
  p.q_pitch = a_scales_stride;
  p.p_shift = shift_of(b_block_rows);
  p.q_shift = shift_of(a_block_rows);
  p.p_rows = (unsigned)n;
  p.q_rows = (unsigned)m;
  p.kblocks = (unsigned)kblocks;
  p.c = c;
  p.c_stride = c_stride;
  p.out_bf16 = c_dtype == XP_BF16;
  p.accumulate = accumulate != 0;
  p.limit_ns = xp::spin_timeout_ns();
  XP_CUDA(xp::launch_matmul8(p, sms, stream));
  return XP_OK;
}

xp_status xp_matmul8_status(void) {
  unsigned n = 0;
  XP_CUDA(xp::matmul8_stalls(&n));
  if (n) return fail(XP_ERR_TIMEOUT, "%u warps of products gave up a wait", n);
  return XP_OK;
}

xp_status xp_rmsnorm_forward(const void* x, size_t x_stride, const void* residual, size_t residual_stride, const void* gamma, void* added,
                             size_t added_stride, void* y, size_t y_stride, uint8_t* y8, size_t y8_stride, uint8_t* y8_scales,
                             size_t y8_scales_stride, float* rstd, size_t rows, size_t cols, float eps, xp_dtype dtype, xp_dtype wdtype,
                             xp_stream_t stream) {
  xp_status s = check_shape(rows, cols);
  if (s != XP_OK || (s = check_types(dtype, wdtype)) != XP_OK) return s;
  if (cols == 0) return fail(XP_ERR_INVALID, "cols is 0");
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(XP_ERR_INVALID, "eps %g is not a number of 0 or more", eps);
  if ((residual != nullptr) != (added != nullptr) && rows) return fail(XP_ERR_INVALID, "residual and added are given together");
  if (rows == 0) return XP_OK;
  const size_t es = size_of(dtype), ws = size_of(wdtype);
  if ((s = check_matrix("x", x, x_stride, rows, cols, dtype)) != XP_OK) return s;
  if (residual && (s = check_matrix("residual", residual, residual_stride, rows, cols, dtype)) != XP_OK) return s;
  if (added && (s = check_matrix("added", added, added_stride, rows, cols, dtype)) != XP_OK) return s;
  if (y && (s = check_matrix("y", y, y_stride, rows, cols, dtype)) != XP_OK) return s;
  if (y8 && (s = check_block8("y8", y8, y8_stride, y8_scales, y8_scales_stride, rows, cols, 1)) != XP_OK) return s;
  if (!aligned(gamma, ws) || !aligned(rstd, 4)) return fail(XP_ERR_INVALID, "gamma or rstd is not aligned to its element");
  const Span sx = span_of(x, x_stride, rows, cols, es);
  Span read[3] = {sx}, written[5];
  size_t nr = 1, nw = 0;
  if (residual) read[nr++] = span_of(residual, residual_stride, rows, cols, es);
  const size_t inputs = nr;
  if (gamma) read[nr++] = span_of(gamma, cols, 1, cols, ws);
  if (added) written[nw++] = span_of(added, added_stride, rows, cols, es);
  if (y) written[nw++] = span_of(y, y_stride, rows, cols, es);
  const size_t in_place = nw;   // these may be an input itself
  if (y8) written[nw++] = span8(y8, y8_stride, rows, cols), written[nw++] = span_scales(y8_scales, y8_scales_stride, rows, cols, 1);
  if (rstd) written[nw++] = span_of(rstd, rows, 1, rows, 4);
  for (size_t i = 0; i < nw; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return fail(XP_ERR_INVALID, "two of added, y, y8, its scales and rstd overlap");
    for (size_t j = 0; j < nr; ++j)
      if (overlap(written[i], read[j]) && !(i < in_place && j < inputs && same(written[i], read[j])))
        return fail(XP_ERR_INVALID, "an output overlaps x, residual or gamma");
  }
  xp::RmsForwardParams p = {};
  p.x = x;
  p.residual = residual;
  p.gamma = gamma;
  p.added = added;
  p.y = y;
  p.y8 = y8;
  p.y8_scales = y8_scales;
  p.rstd = rstd;
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.added_stride = added_stride;
  p.y_stride = y_stride;
  p.y8_stride = y8_stride;
  p.y8_scales_stride = y8_scales_stride;
  p.rows = rows;
  p.cols = (unsigned)cols;
  p.eps = eps;
  p.gamma_bf16 = wdtype == XP_BF16;
  const bool wide = cols * es % 16 == 0 && rows_aligned(x, x_stride, rows, es, 16) && rows_aligned(residual, residual_stride, rows, es, 16) &&
                    rows_aligned(added, added_stride, rows, es, 16) && rows_aligned(y, y_stride, rows, es, 16) && aligned(gamma, 16) &&
                    rows_aligned(y8, y8_stride, rows, 1, 8);
  XP_CUDA(xp::launch_rms_forward(p, dtype, wide, stream));
  return XP_OK;
}

xp_status xp_rmsnorm_workspace(size_t rows, size_t cols, size_t* bytes) {
  if (!bytes) return fail(XP_ERR_INVALID, "bytes is NULL");
  const xp_status s = check_shape(rows, cols);
  if (s != XP_OK) return s;
  *bytes = rows && cols ? rms_workspace(rows, cols, sm_count()) : 0;
  return XP_OK;
}

xp_status xp_rmsnorm_backward(const void* dy, size_t dy_stride, const void* h, size_t h_stride, const void* gamma, const float* rstd,
                              const void* dadded, size_t dadded_stride, void* dx, size_t dx_stride, float* dgamma, size_t rows, size_t cols,
                              xp_dtype dtype, xp_dtype wdtype, int accumulate, void* workspace, size_t workspace_bytes, xp_stream_t stream) {
  xp_status s = check_shape(rows, cols);
  if (s != XP_OK || (s = check_types(dtype, wdtype)) != XP_OK) return s;
  if (cols == 0) return fail(XP_ERR_INVALID, "cols is 0");
  const size_t es = size_of(dtype), ws = size_of(wdtype);
  if (!aligned(gamma, ws) || !aligned(rstd, 4) || !aligned(dgamma, 4)) return fail(XP_ERR_INVALID, "gamma, rstd or dgamma is not aligned to its element");
  if (rows == 0) {
    if (dgamma && !accumulate) XP_CUDA(cudaMemsetAsync(dgamma, 0, cols * sizeof(float), stream));
    return XP_OK;
  }
  if ((s = check_matrix("dy", dy, dy_stride, rows, cols, dtype)) != XP_OK || (s = check_matrix("h", h, h_stride, rows, cols, dtype)) != XP_OK ||
      (s = check_matrix("dx", dx, dx_stride, rows, cols, dtype)) != XP_OK)
    return s;
  if (dadded && (s = check_matrix("dadded", dadded, dadded_stride, rows, cols, dtype)) != XP_OK) return s;
  if (!rstd) return fail(XP_ERR_INVALID, "rstd is NULL");
  const int sms = sm_count();
  const bool wide = cols * es % 16 == 0 && rows_aligned(dy, dy_stride, rows, es, 16) && rows_aligned(h, h_stride, rows, es, 16) &&
                    rows_aligned(dadded, dadded_stride, rows, es, 16) && rows_aligned(dx, dx_stride, rows, es, 16) && aligned(gamma, 16);
  const xp::RmsBackwardShape shape = xp::rms_backward_shape(rows, cols, dtype, wide, sms);
  const bool needed = dgamma || shape.is_long;
  if (needed && workspace_bytes < rms_workspace(rows, cols, sms)) return fail(XP_ERR_INVALID, "workspace of %zu bytes, %zu are needed", workspace_bytes, rms_workspace(rows, cols, sms));
  if (needed && (!workspace || !aligned(workspace, 16))) return fail(XP_ERR_INVALID, "workspace is NULL or not 16-byte aligned");
  const Span sdy = span_of(dy, dy_stride, rows, cols, es), sdx = span_of(dx, dx_stride, rows, cols, es);
  Span read[5] = {sdy, span_of(h, h_stride, rows, cols, es), span_of(rstd, rows, 1, rows, 4)}, written[3] = {sdx};
  size_t nr = 3, nw = 1;
  if (dadded) read[nr++] = span_of(dadded, dadded_stride, rows, cols, es);
  if (gamma) read[nr++] = span_of(gamma, cols, 1, cols, ws);
  if (dgamma) written[nw++] = span_of(dgamma, cols, 1, cols, 4);
  if (needed) written[nw++] = span_of(workspace, workspace_bytes, 1, workspace_bytes, 1);
  for (size_t i = 0; i < nw; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return fail(XP_ERR_INVALID, "two of dx, dgamma and workspace overlap");
    for (size_t j = 0; j < nr; ++j)
      if (overlap(written[i], read[j]) && !(i == 0 && (j == 0 || (j == 3 && dadded)) && same(written[i], read[j])))
        return fail(XP_ERR_INVALID, "dx, dgamma or workspace overlaps an input");
  }
  xp::RmsBackwardParams p = {};
  p.dy = dy;
  p.h = h;
  p.gamma = gamma;
  p.dadded = dadded;
  p.dx = dx;
  p.rstd = rstd;
  p.dgamma = dgamma;
  p.row_sums = static_cast<float*>(workspace);
  p.partial = dgamma ? reinterpret_cast<float*>(static_cast<char*>(workspace) + (shape.is_long ? round_up(rows * 4, 16) : 0)) : nullptr;
  p.dy_stride = dy_stride;
  p.h_stride = h_stride;
  p.dadded_stride = dadded_stride;
  p.dx_stride = dx_stride;
  p.rows = rows;
  p.cols = (unsigned)cols;
  p.gamma_bf16 = wdtype == XP_BF16;
  p.accumulate = accumulate != 0;
  XP_CUDA(xp::launch_rms_backward(p, shape, dtype, wide, stream));
  return XP_OK;
}

xp_status xp_distill_forward(const void* logits, size_t logits_stride, const int32_t* ids, const float* teacher, size_t rows, size_t vocab,
                             size_t top, float temperature, float* loss, float* lse, xp_dtype dtype, xp_stream_t stream) {
  xp_status s = check_distill(logits, logits_stride, ids, teacher, rows, vocab, top, temperature, dtype);
  if (s != XP_OK || rows == 0) return s;
  if (!loss || !aligned(loss, 4) || !aligned(lse, 4)) return fail(XP_ERR_INVALID, "loss is NULL, or loss or lse is not aligned to its element");
  Span read[3] = {span_of(logits, logits_stride, rows, vocab, size_of(dtype))}, written[2] = {span_of(loss, rows, 1, rows, 4)};
  size_t nr = 1, nw = 1;
  if (top) read[nr++] = span_of(ids, top, 1, rows * top, 4), read[nr++] = span_of(teacher, top, 1, rows * top, 4);
  if (lse) written[nw++] = span_of(lse, rows, 1, rows, 4);
  if (any_overlap(written, nw, read, nr)) return fail(XP_ERR_INVALID, "loss or lse overlaps another buffer");
  xp::DistillParams p = {};
  p.logits = logits;
  p.ids = ids;
  p.teacher = teacher;
  p.loss = loss;
  p.lse = lse;
  p.logits_stride = logits_stride;
  p.rows = (unsigned)rows;
  p.vocab = (unsigned)vocab;
  p.top = (unsigned)top;
  p.temperature = temperature;
  XP_CUDA(xp::launch_distill_forward(p, dtype, sm_count(), stream));
  return XP_OK;
}

xp_status xp_distill_backward(const void* logits, size_t logits_stride, const int32_t* ids, const float* teacher, const float* lse,
                              const float* dloss, size_t rows, size_t vocab, size_t top, float temperature, void* dlogits,
                              size_t dlogits_stride, xp_dtype dtype, xp_stream_t stream) {
  xp_status s = check_distill(logits, logits_stride, ids, teacher, rows, vocab, top, temperature, dtype);
  if (s != XP_OK || rows == 0) return s;
  if ((s = check_matrix("dlogits", dlogits, dlogits_stride, rows, vocab, dtype)) != XP_OK) return s;
  if (!lse || !dloss || !aligned(lse, 4) || !aligned(dloss, 4)) return fail(XP_ERR_INVALID, "lse or dloss is NULL or not aligned to its element");
  const size_t es = size_of(dtype);
  const Span z = span_of(logits, logits_stride, rows, vocab, es), dz = span_of(dlogits, dlogits_stride, rows, vocab, es), written[1] = {dz};
  Span read[5] = {span_of(lse, rows, 1, rows, 4), span_of(dloss, rows, 1, rows, 4)};
  size_t nr = 2;
  if (top) read[nr++] = span_of(ids, top, 1, rows * top, 4), read[nr++] = span_of(teacher, top, 1, rows * top, 4);
  if (!same(z, dz)) read[nr++] = z;
  if (any_overlap(written, 1, read, nr)) return fail(XP_ERR_INVALID, "dlogits overlaps another buffer");
  xp::DistillParams p = {};
  p.logits = logits;
  p.ids = ids;
  p.teacher = teacher;
  p.lse = const_cast<float*>(lse);
  p.dloss = dloss;
  p.dlogits = dlogits;
  p.logits_stride = logits_stride;
  p.dlogits_stride = dlogits_stride;
  p.rows = (unsigned)rows;
  p.vocab = (unsigned)vocab;
  p.top = (unsigned)top;
  p.temperature = temperature;
  XP_CUDA(xp::launch_distill_backward(p, dtype, sm_count(), stream));
  return XP_OK;
}

}  // extern "C"
