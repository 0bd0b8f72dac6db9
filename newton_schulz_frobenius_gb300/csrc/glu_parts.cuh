// What the feed-forward block's kernels (glu.cu) and the experts' products
// (expert_products.cu) share: the activations, the preparation of operands and
// of dG and dU in one launch, and the tensor maps of 16-bit matrices.
#pragma once

#include "host.h"
#include "tc_ptx.cuh"

namespace muon {

enum Act : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// act(g), and act'(g) where asked for.  Written so that large finite |g| give 0,
// 1 or g, never an infinity times zero.
template <bool GRAD>
__device__ __forceinline__ float activate(float g, int act, float* grad) {
    if (act == ACT_GELU) {
        const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
        if (GRAD) *grad = fmaf(g * expf(-0.5f * g * g), 0.3989422804014327f, cdf);
        return g * cdf;
    }
    if (act == ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = sigmoid(2 u)
        const float k2 = 1.5957691216057308f;
        const float s = 1.0f / (1.0f + __expf(-k2 * g * fmaf(0.044715f * g, g, 1.0f)));
        if (GRAD) {
            const float c = fminf(fmaxf(g, -30.f), 30.f);
            *grad = fmaf(c * s * (1.0f - s), k2 * fmaf(0.134145f * c, c, 1.0f), s);
        }
        return g * s;
    }
    const float s = 1.0f / (1.0f + __expf(-g));
    if (GRAD) *grad = s * fmaf(g, 1.0f - s, 1.0f);
    return g * s;
}

// One output matrix: rows x cols, row-major with pitch ld.
struct GluOut {
    void* p;
    int64_t ld;
};

// dG = dH U act'(G) and dU = dH act(G) over dense rows x ffn matrices, written at
// a pitch of whole 16-byte pieces (zeros beyond ffn).  Computed in fp32 and rounded
// to 16 bits, what the tensor core takes as operands: the gradients' error against 64
// bits is 0.0023 of their norm in bf16 (fp16 0.00029) where their own rounding alone
// leaves 0.0017 (0.00021); two 16-bit terms each would double the products.
struct GluGradArgs {
    const void* dh;
    const void* gate;
    const void* up;
    void* dg;
    void* du;
    int64_t rows;
    int ffn, pieces;            // columns, 16-byte pieces of a workspace row
    int dtype, act;
    int vec;                    // the inputs' rows start on 16 bytes too
};

struct Operand {
    const void* p;
    int64_t rows, cols, ld;
};

inline bool tma_ok(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

// A caller's matrix as the copy engine can read it: itself, or (rows that do not
// start on 16 bytes) a padded copy at `at` in the workspace.
inline size_t padded_bytes(const Operand& o) {
    return tma_ok(o.p, o.ld) ? 0 : align_up((size_t)o.rows * pad8(o.cols) * 2, 256);
}

// Points those of the dense block's three operands (ops; null: none) that need it at
// padded copies and makes these, with dG and dU where `g` is given, in one launch
// (glu.cu).  The experts' operands, of different widths and counts, have a kernel of
// their own.
int glu_prepare(Operand* const* ops, char* at, const GluGradArgs* g, int sms, cudaStream_t s);

// `batch` matrices of o.rows x o.cols, one after the other (o.rows * o.ld apart).
inline bool map_in(CUtensorMap* m, const Operand& o, int dtype, uint32_t box_cols, uint32_t box_rows, int64_t batch = 1) {
    return tc::make_map(m, o.p, dtype, (uint64_t)o.cols, (uint64_t)o.rows, (uint64_t)batch, (uint64_t)o.ld,
                        (uint64_t)(o.rows * o.ld), box_cols, box_rows);
}

// Chunks of 32 columns (64-byte swizzled) and 32 or 16 rows.
inline bool map_out(CUtensorMap* m, const GluOut& o, int dtype, int64_t rows, int64_t cols, int64_t batch = 1,
                    uint32_t box_rows = 32) {
    auto fn = tc::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.ld * 2 * (cuuint64_t)rows};
    cuuint32_t box[3] = {32, box_rows, 1}, elem[3] = {1, 1, 1};
    return fn(m, dtype == MUON_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, o.p, dims,
              strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace muon
