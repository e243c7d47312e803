// The C-ABI boundary of the linear layer's operators: argument checks and
// dispatch to the kernel launchers.  Host only; an argument error makes no
// CUDA call.
#include "tr_internal.h"

#include <cmath>

namespace tr {
namespace {

int esize_of(int32_t dtype) {
    return dtype == TR_DTYPE_F32 ? 4 : dtype == TR_DTYPE_BF16 ? 2 : 1;
}
bool wide(int32_t dtype) { return dtype == TR_DTYPE_F32 || dtype == TR_DTYPE_BF16; }
bool narrow(int32_t dtype) { return dtype == TR_DTYPE_E4M3 || dtype == TR_DTYPE_E5M2; }
int64_t blocks_of(int64_t n, int64_t block) { return n / block + (n % block != 0); }

// The byte range of one operand; `first` == `last` where it holds nothing.
struct Range {
    uintptr_t first, last;
};

// Checks one rows x cols operand at pitch ld and fills its range: not NULL, on
// its `align` boundary, pitch at least cols, extent within int64 and the
// address space.
tr_status side_range(const void *p, int64_t rows, int64_t cols, int64_t ld, int esize, int align,
                     Range *r) {
    *r = Range{0, 0};
    if (rows == 0 || cols == 0) return TR_OK;
    if (!p) return TR_ERR_NULL;
    if (ld < cols) return TR_ERR_BAD_LD;
    int64_t ext, bytes;
    if (!mul_add(rows - 1, ld, cols, &ext) || !mul_add(ext, esize, 0, &bytes)) return TR_ERR_BAD_DIM;
    r->first = reinterpret_cast<uintptr_t>(p);
    r->last = r->first + uintptr_t(bytes);
    if (r->last < r->first) return TR_ERR_BAD_DIM;
    if (r->first % uintptr_t(align)) return TR_ERR_UNSUPPORTED;
    return TR_OK;
}

bool overlap(const Range &a, const Range &b) {
    return a.first != a.last && b.first != b.last && a.first < b.last && b.first < a.last;
}

// Whether any of the outputs touches an input or another output.
bool outputs_overlap(const Range *out, int n_out, const Range *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

tr_status cuda_status(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return TR_OK;
    set_error(what, e);
    return TR_ERR_CUDA;
}

tr_status unsupported(const char *why) {
    set_error(why, cudaSuccess);
    return TR_ERR_UNSUPPORTED;
}

#define TR_TRY(call)                               \
    do {                                           \
        const tr_status st_ = (call);              \
        if (st_ != TR_OK) return st_;              \
    } while (0)

tr_status quantize(const tr_quantize_args *a) {
    if (!a) return TR_ERR_NULL;
    if (a->reserved != 0 || !wide(a->x_dtype) || !narrow(a->q_dtype) ||
        (a->block_rows != 1 && a->block_rows != 128))
        return unsupported("quantize: fp32 or bf16 to an 8-bit type, block_rows 1 or 128");
    if (a->rows < 0 || a->cols < 0) return TR_ERR_BAD_DIM;
    if (a->rows == 0 || a->cols == 0) return TR_OK;
    const int64_t b = a->block_rows;
    Range in, out[4] = {};
    TR_TRY(side_range(a->x, a->rows, a->cols, a->ld_x, esize_of(a->x_dtype), esize_of(a->x_dtype), &in));
    TR_TRY(side_range(a->q, a->rows, a->cols, a->ld_q, 1, 16, &out[0]));
    TR_TRY(side_range(a->scale, blocks_of(a->cols, 128), blocks_of(a->rows, b), a->ld_scale, 4, 4, &out[1]));
    if (a->ld_q % 16) return unsupported("quantize: ld_q must be a multiple of 16");
    if (a->qt) {
        TR_TRY(side_range(a->qt, a->cols, a->rows, a->ld_qt, 1, 16, &out[2]));
        TR_TRY(side_range(a->scale_t, blocks_of(a->rows, 128), blocks_of(a->cols, b), a->ld_scale_t, 4, 4, &out[3]));
        if (a->ld_qt % 16) return unsupported("quantize: ld_qt must be a multiple of 16");
    }
    if (outputs_overlap(out, 4, &in, 1)) return TR_ERR_OVERLAP;
    return cuda_status("quantize launch failed", launch_quantize(*a));
}

tr_status matmul_fp8(const tr_matmul_fp8_args *a) {
    if (!a) return TR_ERR_NULL;
    if (!narrow(a->a_dtype) || !narrow(a->b_dtype) || !wide(a->out_dtype) ||
        (a->a_block_rows != 1 && a->a_block_rows != 128) ||
        (a->b_block_rows != 1 && a->b_block_rows != 128) || (a->accumulate & ~1))
        return unsupported("matmul: 8-bit operands, fp32 or bf16 out, block rows 1 or 128, accumulate 0 or 1");
    if (a->m < 0 || a->n < 0 || a->k < 0) return TR_ERR_BAD_DIM;
    if (a->m == 0 || a->n == 0) return TR_OK;
    const int64_t top = int64_t(1) << 31;
    if (a->m >= top || a->n >= top || a->k >= top)
        return unsupported("matmul: a dimension is 2^31 or more");
    const int64_t kb = blocks_of(a->k, 128);
    Range in[4], out;
    TR_TRY(side_range(a->out, a->m, a->n, a->ld_out, esize_of(a->out_dtype), esize_of(a->out_dtype), &out));
    TR_TRY(side_range(a->a, a->m, a->k, a->lda, 1, 16, &in[0]));
    TR_TRY(side_range(a->b, a->n, a->k, a->ldb, 1, 16, &in[1]));
    TR_TRY(side_range(a->scale_a, kb, blocks_of(a->m, a->a_block_rows), a->ld_scale_a, 4, 4, &in[2]));
    TR_TRY(side_range(a->scale_b, kb, blocks_of(a->n, a->b_block_rows), a->ld_scale_b, 4, 4, &in[3]));
    if (a->k && (a->lda % 16 || a->ldb % 16))
        return unsupported("matmul: lda and ldb must be multiples of 16");
    if (outputs_overlap(&out, 1, in, 4)) return TR_ERR_OVERLAP;
    const char *why = nullptr;
    const cudaError_t e = launch_matmul_fp8(*a, &why);
    if (e != cudaSuccess && why) return unsupported(why);
    return cuda_status("matmul launch failed", e);
}

tr_status layernorm(const tr_layernorm_args *a) {
    if (!a) return TR_ERR_NULL;
    if (a->reserved != 0 || !wide(a->x_dtype) || !wide(a->w_dtype))
        return unsupported("layer norm: fp32 or bf16");
    if (a->rows < 0 || a->cols < 0 || !(a->eps >= 0) || std::isinf(a->eps)) return TR_ERR_BAD_DIM;
    if (a->rows == 0 || a->cols == 0) return TR_OK;
    const int es = esize_of(a->x_dtype), ws = esize_of(a->w_dtype);
    Range in[3] = {}, out[3] = {};
    TR_TRY(side_range(a->x, a->rows, a->cols, a->ld_x, es, es, &in[0]));
    TR_TRY(side_range(a->gamma, 1, a->cols, a->cols, ws, ws, &in[1]));
    if (a->beta) TR_TRY(side_range(a->beta, 1, a->cols, a->cols, ws, ws, &in[2]));
    TR_TRY(side_range(a->y, a->rows, a->cols, a->ld_y, es, es, &out[0]));
    if (a->mean) TR_TRY(side_range(a->mean, 1, a->rows, a->rows, 4, 4, &out[1]));
    if (a->rstd) TR_TRY(side_range(a->rstd, 1, a->rows, a->rows, 4, 4, &out[2]));
    if (outputs_overlap(out, 3, in, 3)) return TR_ERR_OVERLAP;
    return cuda_status("layer norm launch failed", launch_layernorm(*a));
}

tr_status layernorm_backward(const tr_layernorm_backward_args *a) {
    if (!a) return TR_ERR_NULL;
    if (!wide(a->x_dtype) || !wide(a->w_dtype)) return unsupported("layer norm: fp32 or bf16");
    if (a->rows < 0 || a->cols < 0) return TR_ERR_BAD_DIM;
    if (a->cols == 0) return TR_OK;
    const int es = esize_of(a->x_dtype), ws = esize_of(a->w_dtype);
    const int64_t need = tr_layernorm_backward_workspace(a->rows, a->cols);
    if (need < 0) return TR_ERR_BAD_DIM;
    Range in[5] = {}, out[4] = {};
    TR_TRY(side_range(a->dgamma, 1, a->cols, a->cols, 4, 4, &out[0]));
    if (a->dbeta) TR_TRY(side_range(a->dbeta, 1, a->cols, a->cols, 4, 4, &out[1]));
    if (a->rows) {
        TR_TRY(side_range(a->dy, a->rows, a->cols, a->ld_dy, es, es, &in[0]));
        TR_TRY(side_range(a->x, a->rows, a->cols, a->ld_x, es, es, &in[1]));
        TR_TRY(side_range(a->gamma, 1, a->cols, a->cols, ws, ws, &in[2]));
        TR_TRY(side_range(a->mean, 1, a->rows, a->rows, 4, 4, &in[3]));
        TR_TRY(side_range(a->rstd, 1, a->rows, a->rows, 4, 4, &in[4]));
        TR_TRY(side_range(a->dx, a->rows, a->cols, a->ld_dx, es, es, &out[2]));
        if (a->workspace_bytes < need) return unsupported("layer norm: the workspace is too small");
        TR_TRY(side_range(a->workspace, 1, need, need, 1, 16, &out[3]));
    }
    if (outputs_overlap(out, 4, in, 5)) return TR_ERR_OVERLAP;
    return cuda_status("layer norm backward launch failed", launch_layernorm_backward(*a));
}

// The same operand twice over, of the same size: what an output may share with the input that it
// replaces.
bool same_side(const void *a, int64_t ld_a, const void *b, int64_t ld_b) { return a == b && ld_a == ld_b; }

tr_status rmsnorm(const tr_rmsnorm_args *a) {
    if (!a) return TR_ERR_NULL;
    if (a->reserved != 0 || a->reserved2 != 0 || !wide(a->x_dtype) || !wide(a->w_dtype))
        return unsupported("rms norm: fp32 or bf16");
    if (a->q && !narrow(a->q_dtype)) return unsupported("rms norm: q is of an 8-bit type");
    if (a->rows < 0 || a->cols < 0 || !(a->eps >= 0) || std::isinf(a->eps)) return TR_ERR_BAD_DIM;
    if (a->rows == 0 || a->cols == 0) return TR_OK;
    if (a->residual ? !a->h : a->h != nullptr)
        return a->residual ? TR_ERR_NULL : unsupported("rms norm: without a residual h is x, and not written");
    if (a->qt && (!a->q || !a->rstd)) return TR_ERR_NULL;
    const int es = esize_of(a->x_dtype), ws = esize_of(a->w_dtype);
    const int64_t cb = blocks_of(a->cols, 128), rb = blocks_of(a->rows, 128);
    Range in[3] = {}, out[7] = {};
    TR_TRY(side_range(a->x, a->rows, a->cols, a->ld_x, es, es, &in[0]));
    TR_TRY(side_range(a->gamma, 1, a->cols, a->cols, ws, ws, &in[1]));
    if (a->residual) {
        TR_TRY(side_range(a->residual, a->rows, a->cols, a->ld_residual, es, es, &in[2]));
        TR_TRY(side_range(a->h, a->rows, a->cols, a->ld_h, es, es, &out[0]));
        if (same_side(a->residual, a->ld_residual, a->h, a->ld_h)) in[2] = Range{0, 0};
    }
    if (a->y) TR_TRY(side_range(a->y, a->rows, a->cols, a->ld_y, es, es, &out[1]));
    if (a->rstd) TR_TRY(side_range(a->rstd, 1, a->rows, a->rows, 4, 4, &out[2]));
    if (a->q) {
        TR_TRY(side_range(a->q, a->rows, a->cols, a->ld_q, 1, 16, &out[3]));
        TR_TRY(side_range(a->scale, cb, a->rows, a->ld_scale, 4, 4, &out[4]));
        if (a->ld_q % 16) return unsupported("rms norm: ld_q must be a multiple of 16");
    }
    if (a->qt) {
        TR_TRY(side_range(a->qt, a->cols, a->rows, a->ld_qt, 1, 16, &out[5]));
        TR_TRY(side_range(a->scale_t, rb, a->cols, a->ld_scale_t, 4, 4, &out[6]));
        if (a->ld_qt % 16) return unsupported("rms norm: ld_qt must be a multiple of 16");
    }
    if (outputs_overlap(out, 7, in, 3)) return TR_ERR_OVERLAP;
    return cuda_status("rms norm launch failed", launch_rmsnorm(*a));
}

tr_status rmsnorm_backward(const tr_rmsnorm_backward_args *a) {
    if (!a) return TR_ERR_NULL;
    if (!wide(a->x_dtype) || !wide(a->w_dtype)) return unsupported("rms norm: fp32 or bf16");
    if (a->rows < 0 || a->cols < 0) return TR_ERR_BAD_DIM;
    if (a->cols == 0) return TR_OK;
    const int es = esize_of(a->x_dtype), ws = esize_of(a->w_dtype);
    const int64_t need = tr_rmsnorm_backward_workspace(a->rows, a->cols);
    if (need < 0) return TR_ERR_BAD_DIM;
    Range in[5] = {}, out[3] = {};
    TR_TRY(side_range(a->dgamma, 1, a->cols, a->cols, 4, 4, &out[0]));
    if (a->rows) {
        TR_TRY(side_range(a->dy, a->rows, a->cols, a->ld_dy, es, es, &in[0]));
        TR_TRY(side_range(a->h, a->rows, a->cols, a->ld_h, es, es, &in[1]));
        TR_TRY(side_range(a->gamma, 1, a->cols, a->cols, ws, ws, &in[2]));
        TR_TRY(side_range(a->rstd, 1, a->rows, a->rows, 4, 4, &in[3]));
        if (a->dresidual) TR_TRY(side_range(a->dresidual, a->rows, a->cols, a->ld_dresidual, es, es, &in[4]));
        TR_TRY(side_range(a->dx, a->rows, a->cols, a->ld_dx, es, es, &out[1]));
        if (a->dresidual && same_side(a->dresidual, a->ld_dresidual, a->dx, a->ld_dx)) in[4] = Range{0, 0};
        if (a->workspace_bytes < need) return unsupported("rms norm: the workspace is too small");
        TR_TRY(side_range(a->workspace, 1, need, need, 1, 16, &out[2]));
    }
    if (outputs_overlap(out, 3, in, 5)) return TR_ERR_OVERLAP;
    return cuda_status("rms norm backward launch failed", launch_rmsnorm_backward(*a));
}

tr_status adapter_plan(const tr_adapter_plan_args *a) {
    if (!a) return TR_ERR_NULL;
    if (a->tokens < 0 || a->adapters < 0) return TR_ERR_BAD_DIM;
    const int64_t need = tr_adapter_plan_bytes(a->tokens, a->adapters);
    if (need < 0) return unsupported("adapters: 2^31 tokens or 2^15 adapters, or more");
    if (a->tokens == 0) return TR_OK;
    Range in, out;
    TR_TRY(side_range(a->index, 1, a->tokens, a->tokens, 4, 4, &in));
    if (a->plan_bytes < need) return unsupported("adapters: the plan is too small");
    TR_TRY(side_range(a->plan, 1, need, need, 1, 16, &out));
    if (overlap(in, out)) return TR_ERR_OVERLAP;
    return cuda_status("adapter plan launch failed", launch_adapter_plan(*a));
}

// Planes of rows x cols at a stride: as side_range, with rows, pitch and stride on 16-byte boundaries.
tr_status planes_range(const void *p, int64_t planes, int64_t rows, int64_t cols, int64_t ld, int64_t stride, Range *r) {
    *r = Range{0, 0};
    if (planes == 0 || rows == 0 || cols == 0) return TR_OK;
    Range plane;
    TR_TRY(side_range(p, rows, cols, ld, 2, 16, &plane));
    int64_t bytes;
    if (stride < 0 || (planes > 1 && stride < int64_t(plane.last - plane.first) / 2)) return TR_ERR_BAD_LD;
    if (!mul_add(planes - 1, stride, int64_t(plane.last - plane.first) / 2, &bytes) || !mul_add(bytes, 2, 0, &bytes))
        return TR_ERR_BAD_DIM;
    *r = Range{plane.first, plane.first + uintptr_t(bytes)};
    if (r->last < r->first) return TR_ERR_BAD_DIM;
    if (ld % 8 || (planes > 1 && stride % 8)) return unsupported("adapters: pitches and strides of x, a and b must be multiples of 8");
    return TR_OK;
}

tr_status adapters(const tr_adapters_args *a) {
    if (!a) return TR_ERR_NULL;
    if (a->reserved != 0 || !wide(a->out_dtype)) return unsupported("adapters: fp32 or bf16 out");
    if (a->tokens < 0 || a->adapters < 0 || a->k < 0 || a->n < 0) return TR_ERR_BAD_DIM;
    const int64_t top = int64_t(1) << 30, need = tr_adapter_plan_bytes(a->tokens, a->adapters);
    if (a->rank < 1 || a->rank > 128) return unsupported("adapters: ranks are 1 to 128");
    if (need < 0 || a->k >= top || a->n >= top) return unsupported("adapters: 2^31 tokens, 2^30 values to a row or 2^15 adapters, or more");
    if (a->tokens == 0 || a->n == 0) return TR_OK;
    const int es = esize_of(a->out_dtype);
    Range in[6] = {}, out;
    TR_TRY(planes_range(a->x, 1, a->tokens, a->k, a->ld_x, 0, &in[0]));
    TR_TRY(planes_range(a->a, a->adapters, a->rank, a->k, a->ld_a, a->stride_a, &in[1]));
    TR_TRY(planes_range(a->b, a->adapters, a->n, a->rank, a->ld_b, a->stride_b, &in[2]));
    if (a->scale) TR_TRY(side_range(a->scale, 1, a->adapters, a->adapters, 4, 4, &in[3]));
    if (a->plan_bytes < need) return unsupported("adapters: the plan is too small");
    TR_TRY(side_range(a->plan, 1, need, need, 1, 16, &in[4]));
    if (a->base) TR_TRY(side_range(a->base, a->tokens, a->n, a->ld_base, es, es, &in[5]));
    TR_TRY(side_range(a->out, a->tokens, a->n, a->ld_out, es, es, &out));
    if (a->base && same_side(a->base, a->ld_base, a->out, a->ld_out)) in[5] = Range{0, 0};
    if (outputs_overlap(&out, 1, in, 6)) return TR_ERR_OVERLAP;
    const char *why = nullptr;
    const cudaError_t e = launch_adapters(*a, &why);
    if (e != cudaSuccess && why) return unsupported(why);
    return cuda_status("adapters launch failed", e);
}

}  // namespace
}  // namespace tr

extern "C" {

tr_status tr_quantize_fp8(const tr_quantize_args *args) { return tr::quantize(args); }

tr_status tr_matmul_fp8(const tr_matmul_fp8_args *args) { return tr::matmul_fp8(args); }

tr_status tr_layernorm(const tr_layernorm_args *args) { return tr::layernorm(args); }

tr_status tr_layernorm_backward(const tr_layernorm_backward_args *args) {
    return tr::layernorm_backward(args);
}

tr_status tr_rmsnorm(const tr_rmsnorm_args *args) { return tr::rmsnorm(args); }

tr_status tr_rmsnorm_backward(const tr_rmsnorm_backward_args *args) { return tr::rmsnorm_backward(args); }

tr_status tr_adapter_plan(const tr_adapter_plan_args *args) { return tr::adapter_plan(args); }

tr_status tr_adapters(const tr_adapters_args *args) { return tr::adapters(args); }

}  // extern "C"
