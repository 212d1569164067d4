// channel_desc.cpp -- matrix descriptors of the channel operators and their
// host-side checks.
#include "channel.h"

namespace i8c {

MatRef mat_ref(const conv_matrix_desc *d, const void *p) {
    MatRef m;
    if (!d) return m;
    m.p = p;
    m.rs = d->rows > 1 ? d->row_stride : 0;
    m.cs = d->cols > 1 ? d->col_stride : 0;
    m.dtype = d->dtype;
    return m;
}

uint64_t matrix_extent_bytes(const conv_matrix_desc *d) {
    if (d->rows == 0 || d->cols == 0) return 0;
    const int64_t rs = d->rows > 1 ? d->row_stride : 0, cs = d->cols > 1 ? d->col_stride : 0;
    return (uint64_t)((d->rows - 1) * rs + (d->cols - 1) * cs + 1) * (uint64_t)channel_elem_size(d->dtype);
}

conv_status check_matrix(const conv_matrix_desc *d) {
    if (!d) return CONV_ERR_NULL_PTR;
    if (d->dtype < CONV_INT8 || d->dtype > CONV_FLOAT8_E5M2) return CONV_ERR_DTYPE;
    if (d->reserved != 0 || d->rows < 0 || d->cols < 0) return CONV_ERR_BAD_PARAM;
    // tile coordinates are 32-bit, a tile may reach 256 past the extent
    if (d->rows > INT32_MAX - 256 || d->cols > INT32_MAX - 256) return CONV_ERR_TOO_LARGE;
    if (d->rows == 0 || d->cols == 0) return CONV_OK;  // nothing is addressed
    // extents are below 2^31: strides up to 2^30 keep every byte offset in
    // 63 bits
    const int64_t cap = (int64_t)1 << 30;
    if ((d->rows > 1 && d->row_stride > cap * 64) || (d->cols > 1 && d->col_stride > cap * 64))
        return CONV_ERR_TOO_LARGE;
    const int64_t rs = d->rows > 1 ? d->row_stride : 0, cs = d->cols > 1 ? d->col_stride : 0;
    if ((d->rows > 1 && rs < 1) || (d->cols > 1 && cs < 1)) return CONV_ERR_BAD_STRIDES;
    const __int128 row_span = (__int128)(d->rows - 1) * rs, col_span = (__int128)(d->cols - 1) * cs;
    if (d->rows > 1 && d->cols > 1) {
        // the dim with the larger stride steps over the whole other dim
        if (rs >= cs ? (__int128)rs <= col_span : (__int128)cs <= row_span) return CONV_ERR_BAD_STRIDES;
    }
    const __int128 bytes = (row_span + col_span + 1) * channel_elem_size(d->dtype);
    if (bytes > ((__int128)1 << 60)) return CONV_ERR_TOO_LARGE;
    if ((unsigned __int128)bytes > d->capacity_bytes) return CONV_ERR_BUFFER_TOO_SMALL;
    return CONV_OK;
}

conv_status check_address(const conv_matrix_desc *d, const void *p) {
    if (d->rows == 0 || d->cols == 0) return CONV_OK;
    if (!p) return CONV_ERR_NULL_PTR;
    if ((uintptr_t)p % (uintptr_t)channel_elem_size(d->dtype)) return CONV_ERR_ALIGNMENT;
    return CONV_OK;
}

// Rows (lines of `len` bytes every `step` bytes) of two matrices with one
// step: they share no byte if each line of b falls between two lines of a.
static bool lines_interleave(int64_t delta, int64_t step, int64_t a_len, int64_t b_len) {
    int64_t off = delta % step;
    if (off < 0) off += step;
    return a_len <= off && off + b_len <= step;
}

bool matrices_overlap(const conv_matrix_desc *a, const void *a_dev, const conv_matrix_desc *b, const void *b_dev) {
    if (!overlaps(a_dev, matrix_extent_bytes(a), b_dev, matrix_extent_bytes(b))) return false;
    const int64_t ea = channel_elem_size(a->dtype), eb = channel_elem_size(b->dtype);
    const int64_t delta = (int64_t)((uintptr_t)b_dev - (uintptr_t)a_dev);
    const bool a_rows = a->cols <= 1 || a->col_stride == 1, b_rows = b->cols <= 1 || b->col_stride == 1;
    if (a_rows && b_rows && a->rows > 1 && b->rows > 1 && a->row_stride * ea == b->row_stride * eb &&
        lines_interleave(delta, a->row_stride * ea, a->cols * ea, b->cols * eb))
        return false;
    const bool a_cols = a->rows <= 1 || a->row_stride == 1, b_cols = b->rows <= 1 || b->row_stride == 1;
    if (a_cols && b_cols && a->cols > 1 && b->cols > 1 && a->col_stride * ea == b->col_stride * eb &&
        lines_interleave(delta, a->col_stride * ea, a->rows * ea, b->rows * eb))
        return false;
    return true;
}

}  // namespace i8c
