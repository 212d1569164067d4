// channel.h -- declarations shared by the channel operators (matrix product
// with epilogue, layer norm, their gradients).  Not part of the public ABI.
#pragma once

#include "internal.h"

namespace i8c {

// One validated matrix operand: address and element strides of rows and
// columns (0 for a dim of extent 1, so kernels may multiply it freely).
struct MatRef {
    const void *p = nullptr;
    int64_t rs = 0, cs = 0;
    int32_t dtype = 0;
};

MatRef mat_ref(const conv_matrix_desc *d, const void *p);

inline int64_t channel_elem_size(int32_t dtype) {
    return dtype == CONV_INT8 || dtype == CONV_FLOAT8_E4M3 || dtype == CONV_FLOAT8_E5M2 ? 1
           : dtype == CONV_FLOAT16 || dtype == CONV_BFLOAT16                            ? 2
                                                                                         : 4;
}

inline bool is_half_type(int32_t dtype) { return dtype == CONV_FLOAT16 || dtype == CONV_BFLOAT16; }
inline bool is_float_type(int32_t dtype) { return dtype == CONV_FLOAT32 || is_half_type(dtype); }
inline bool is_eight_bit_type(int32_t dtype) { return dtype == CONV_FLOAT8_E4M3 || dtype == CONV_FLOAT8_E5M2; }

constexpr int64_t kScaleBlock = 128;  // elements that share a scale

// Checks one matrix: extents 0..2^31-257, positive strides that alias no two
// elements, extent inside capacity_bytes.  The type is the caller's concern.
conv_status check_matrix(const conv_matrix_desc *d);

// Address given (unless the matrix is empty) and a multiple of the element.
conv_status check_address(const conv_matrix_desc *d, const void *p);

// Whether two matrices share a byte.  Matrices whose byte ranges interleave
// are told apart when they have one row (or column) stride and contiguous
// columns (rows), as column blocks of one buffer do; else they count as
// overlapping.
bool matrices_overlap(const conv_matrix_desc *a, const void *a_dev, const conv_matrix_desc *b, const void *b_dev);
uint64_t matrix_extent_bytes(const conv_matrix_desc *d);
inline bool same_matrix(const conv_matrix_desc *a, const void *a_dev, const conv_matrix_desc *b, const void *b_dev) {
    return a_dev == b_dev && (a->rows <= 1 || a->row_stride == b->row_stride) &&
           (a->cols <= 1 || a->col_stride == b->col_stride);
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// ---------------------------------------------------------------- product
// D[a,b] = epilogue(sum_k A[a,k] * B[b,k]) over 16-bit float operands.
struct ProductOperand {
    const void *p = nullptr;
    int64_t s_mn = 0, s_k = 0;  // element strides along a (or b) and along k
};

struct Product {
    int64_t ma = 0, nb = 0, k = 0;
    ProductOperand a, b;
    int32_t in_dtype = 0;        // CONV_FLOAT16 or CONV_BFLOAT16, both operands
    // output, residual (type of the output) and pre-activation (type of the
    // operands): element strides along a and along b
    void *d = nullptr;
    int64_t d_sa = 0, d_sb = 0;
    int32_t d_dtype = 0;
    const void *res = nullptr;
    int64_t res_sa = 0, res_sb = 0;
    void *pre = nullptr;
    int64_t pre_sa = 0, pre_sb = 0;
    const void *bias = nullptr;  // along b (along a when bias_along_a)
    int32_t bias_dtype = 0;
    bool bias_along_a = false;
    int32_t act = CONV_ACT_NONE;
    // The stream's previous kernel shares no buffer with this product but
    // inputs, and lets its successor start only after all before it has
    // ended: the two may run side by side.
    bool beside_previous = false;
};

// Operand the kernel reads in place: one stride 1, the other a multiple of 8
// elements, the address 16-byte aligned.  (Strides of extents of 1 are 0.)
bool product_in_place(const void *p, int64_t rows, int64_t rs, int64_t cols, int64_t cs);

// Tile shape and split of a product of these extents; part_bytes of workspace
// hold its partial sums.
struct ProductPlan {
    bool swap = false;     // a and b exchanged
    bool pair = false;     // tiles of CTA pairs (256 rows), else of one CTA (128)
    int32_t tile_b = 0;
    int64_t tiles_a = 0, tiles_b = 0;
    int32_t split = 1;     // CTAs of a cluster that share a tile along k
    int32_t parts = 1;     // runs of k, summed apart and joined by a second kernel, ...
    int64_t full = 0;      // ... of the tiles from this one on
    size_t part_bytes = 0; // a multiple of 256
};

// The product of up to four rows of a by CUDA cores (product_rows.cu).
bool product_rows_applies(const Product &pr);
conv_status product_rows_launch(const Product &pr, void *stream);

ProductPlan product_plan(int64_t ma, int64_t nb, int64_t k);

// workspace: part_bytes of the plan.
conv_status product_launch(const Product &pr, void *workspace, void *stream);

// ---------------------------------------------------------------- product of 8-bit operands
// D[a,b] = epilogue(sum over blocks of 128 k of scale_a * scale_b * sum_k A[a,k] * B[b,k]).
struct ScaledOperand {
    const uint8_t *p = nullptr;  // k contiguous, rows 16-byte aligned
    int64_t rs = 0;
    const float *scale = nullptr;
    int64_t s_rs = 0, s_cs = 0;
    int32_t shift = 0;           // rows that share a scale: 1 << shift
    int32_t e5m2 = 0;
};

struct ScaledProduct {
    int64_t ma = 0, nb = 0, k = 0;
    ScaledOperand a, b;
    void *d = nullptr;
    int64_t d_sa = 0, d_sb = 0;
    int32_t d_dtype = 0;
    const void *res = nullptr;   // of D's type
    int64_t res_sa = 0, res_sb = 0;
    void *pre = nullptr;
    int64_t pre_sa = 0, pre_sb = 0;
    int32_t pre_dtype = 0;
    const void *bias = nullptr;  // along b
    int32_t bias_dtype = 0;
    int32_t act = CONV_ACT_NONE;
};

// Tile shape and runs of the tensor-core product (scaled_product.cu);
// part_bytes of workspace hold its partial sums.
struct ScaledPlan {
    bool swap = false;     // a and b exchanged
    int32_t tile_b = 0;
    int64_t tiles_a = 0, tiles_b = 0;
    int32_t parts = 1;     // runs of k, summed apart and joined by a second kernel, ...
    int64_t full = 0;      // ... of the tiles from this one on
    size_t part_bytes = 0;
};
ScaledPlan scaled_plan(int64_t ma, int64_t nb, int64_t k);
conv_status scaled_launch(const ScaledProduct &pr, void *workspace, void *stream);

// A few rows of a (scaled_rows.cu).
bool scaled_rows_applies(int64_t ma, int64_t nb, int64_t k);
conv_status scaled_rows_launch(const ScaledProduct &pr, void *stream);

}  // namespace i8c
