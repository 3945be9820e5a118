// moe_api.cpp - the C ABI of the 8-bit expert layer: validation and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "api_internal.h"
#include "dg_args.h"
#include "fp8_rules.h"
#include "launch.h"
#include "moe_args.h"

using namespace dg;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int elt_of(int32_t t) { return t == DG_F16 ? T_F16 : t == DG_BF16 ? T_BF16 : t == DG_F32 ? T_F32 : -1; }
int elt_bytes(int e) { return e == T_F32 ? 4 : 2; }

// What every call that launches needs: a live handle of the current device.
dg_status device_ready(dg_handle_t h)
{
    if (!api_live(h)) return api_fail(DG_ERR_INVALID_STATE, "handle is NULL or destroyed");
    if (h->device < 0) return api_fail(DG_ERR_INVALID_STATE, "offline handle: nothing is launched");
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != h->device)
        return api_fail(DG_ERR_INVALID_STATE, "the current HIP device is not the handle's device");
    return DG_OK;
}

dg_status launched(hipError_t e)
{
    if (e == hipErrorInvalidConfiguration)
        return api_fail(DG_ERR_UNSUPPORTED, "the problem takes 2^32 work-items or more, one launch's limit");
    return e == hipSuccess ? DG_OK : api_fail(DG_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

dg_status sizes_ok(std::initializer_list<int64_t> sizes)
{
    for (int64_t v : sizes) {
        if (v < 0) return api_fail(DG_ERR_INVALID_ARG, "negative size or leading dimension");
        if (v > FP8_MOST) return api_fail(DG_ERR_UNSUPPORTED, "sizes above 2^31-4096 are not supported");
    }
    return DG_OK;
}

dg_status check_operands(const void *A, int64_t lda, const float *sa, const void *B, int64_t ldb, const float *sb,
                         int64_t K)
{
    if (!A || !B || !sa || !sb) return api_fail(DG_ERR_INVALID_ARG, "A, B and both scale arrays are required");
    if (!aligned(A, 16) || !aligned(B, 16) || lda % 16 || ldb % 16)
        return api_fail(DG_ERR_ALIGNMENT, "A and B: 16-byte aligned pointers and rows");
    if (!aligned(sa, 4) || !aligned(sb, 4)) return api_fail(DG_ERR_ALIGNMENT, "scale arrays are 4-byte aligned");
    if (!rows_fit_32(128, lda, K) || !rows_fit_32(128, ldb, K))
        return api_fail(DG_ERR_UNSUPPORTED, "128 rows of an operand span 4 GiB or more");
    return DG_OK;
}

dg_status check_out(const void *C, int32_t c_type, int &elt)
{
    elt = elt_of(c_type);
    if (elt < 0) return api_fail(DG_ERR_UNSUPPORTED, "the output type is F16, BF16 or F32");
    if (!C) return api_fail(DG_ERR_INVALID_ARG, "C is NULL");
    if (!aligned(C, elt_bytes(elt))) return api_fail(DG_ERR_ALIGNMENT, "C is misaligned for its type");
    return DG_OK;
}

#define DG_TRY(x)                        \
    do {                                 \
        const dg_status s_ = (x);        \
        if (s_ != DG_OK) return s_;      \
    } while (0)

}  // namespace

extern "C" {

dg_status dg_quant_fp8(dg_handle_t h, int64_t rows, int64_t cols, const void *X, int32_t x_type, int64_t x_rows,
                       int64_t ldx, const int32_t *index, int32_t index_div, int32_t transpose, void *codes,
                       int64_t ldq, float *scales, int64_t ld_scale, dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({rows, cols, x_rows}));
        if (ldx < 0 || ldq < 0 || ld_scale < 0) return api_fail(DG_ERR_INVALID_ARG, "negative size or leading dimension");
        const int elt = elt_of(x_type);
        if (elt < 0) return api_fail(DG_ERR_UNSUPPORTED, "X is F16, BF16 or F32");
        if (transpose != 0 && transpose != 1) return api_fail(DG_ERR_INVALID_ARG, "transpose is 0 or 1");
        const int64_t out_cols = transpose ? rows : cols, out_rows = transpose ? cols : rows;
        const int64_t lx = ldx ? ldx : cols, lq = ldq ? ldq : out_cols, ls = ld_scale ? ld_scale : out_rows;
        if (lx < cols || lq < out_cols || ls < out_rows)
            return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        if (index ? index_div < 1 : x_rows < rows)
            return api_fail(DG_ERR_INVALID_ARG, index ? "index_div must be positive" : "X has fewer rows than asked for");
        if (rows == 0 || cols == 0) return DG_OK;
        if ((!X && x_rows > 0) || !codes || !scales) return api_fail(DG_ERR_INVALID_ARG, "X, codes and scales are required");
        if (!aligned(X, elt_bytes(elt)) || !aligned(scales, 4) || !aligned(index, 4))
            return api_fail(DG_ERR_ALIGNMENT, "a pointer is misaligned for its type");
        QuantFp8Args a{};
        a.X = X, a.index = index, a.codes = codes, a.scales = scales;
        a.x_rows = x_rows, a.ldx = lx, a.ldq = lq, a.ld_scale = ls;
        a.rows = (int)rows, a.cols = (int)cols, a.index_div = index ? index_div : 1, a.x_type = elt;
        return launched(launch_quant_fp8(a, transpose != 0, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_quant_fp8");
    }
}

dg_status dg_plan_fp8(dg_handle_t h, int64_t M, int64_t N, int64_t K, dg_plan_info *out)
{
    try {
        if (!api_live(h)) return api_fail(DG_ERR_INVALID_STATE, "handle is NULL or destroyed");
        DG_TRY(sizes_ok({M, N, K}));
        if (!out) return api_fail(DG_ERR_INVALID_ARG, "out is NULL");
        const Fp8Choice c = choose_dense(M, N, K, huge_tile(false, K, K, K));
        const Fp8Shape &s = fp8_shape(c.kernel);
        dg_plan_info i{};
        i.path = s.stream ? DG_PATH_SKINNY : DG_PATH_TILED;
        i.unit = DG_UNIT_MFMA;
        i.mfma_m = i.mfma_n = 16;
        i.mfma_k = i.k_main = FP8_BLOCK;
        i.m_tile = s.bm;
        i.n_tile = s.bn;
        slices(K, c.split, i.k_slice, i.split_k);
        i.n_main = i.k_slice / FP8_BLOCK;
        i.waves_per_wg = s.threads / 64;
        i.grid = (int32_t)std::min<int64_t>(INT32_MAX, ((M + s.bm - 1) / s.bm) * ((N + s.bn - 1) / s.bn) * i.split_k);
        i.workspace_bytes = i.split_k > 1 ? (int64_t)i.split_k * M * N * 4 : 0;
        i.kernel_id = c.kernel;
        std::strncpy(i.kernel_name, s.name, sizeof i.kernel_name - 1);
        *out = i;
        return DG_OK;
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_plan_fp8");
    }
}

dg_status dg_gemm_fp8(dg_handle_t h, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const float *a_scale,
                      int64_t lda_scale, const void *B, int64_t ldb, const float *b_scale, int64_t ldb_scale,
                      int32_t b_block, void *C, int32_t c_type, int64_t ldc, void *workspace, size_t workspace_bytes,
                      dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({M, N, K}));
        if (lda < 0 || ldb < 0 || lda_scale < 0 || ldb_scale < 0 || ldc < 0)
            return api_fail(DG_ERR_INVALID_ARG, "negative size or leading dimension");
        if (b_block != 1 && b_block != FP8_BLOCK)
            return api_fail(DG_ERR_UNSUPPORTED, "b_block is 1 (a scale per row of B) or 128 (per 128 rows)");
        const int64_t la = lda ? lda : K, lb = ldb ? ldb : K, lc = ldc ? ldc : N;
        const int64_t nsb = b_block == 1 ? N : blocks_of(N);
        const int64_t lsa = lda_scale ? lda_scale : M, lsb = ldb_scale ? ldb_scale : nsb;
        if (la < K || lb < K || lc < N || lsa < M || lsb < nsb)
            return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        if (M == 0 || N == 0) return DG_OK;
        Fp8Args a{};
        DG_TRY(check_out(C, c_type, a.out_type));
        if (K > 0) DG_TRY(check_operands(A, la, a_scale, B, lb, b_scale, K));
        const Fp8Choice c = choose_dense(M, N, K, huge_tile(a.out_type == T_F32, la, lb, K));
        slices(K, c.split, a.k_slice, a.split_k);
        if (a.split_k > 1) {
            const size_t need = (size_t)a.split_k * M * N * 4;
            if (!workspace || workspace_bytes < need)
                return api_fail(DG_ERR_WORKSPACE, "workspace missing or smaller than " + std::to_string(need) + " bytes");
            if (!aligned(workspace, 16)) return api_fail(DG_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
        }
        a.A = A, a.B = B, a.sa = a_scale, a.sb = b_scale, a.C = C;
        a.lda = la, a.ldb = lb, a.ld_sa = lsa, a.ld_sb = lsb, a.ldc = lc;
        a.M = (int)M, a.N = (int)N, a.K = (int)K;
        a.ws = reinterpret_cast<float *>(workspace);
        hipStream_t st = reinterpret_cast<hipStream_t>(stream);
        DG_TRY(launched(launch_fp8(c.kernel, FP8_DENSE, b_block, a, st)));
        if (a.split_k > 1) {   // the slices' sums, added in slice order
            ReduceArgs r{};
            r.ws = workspace;
            r.split_k = a.split_k, r.M = (int)M, r.N = (int)N, r.lanes = 1;
            r.epi.C = C, r.epi.ldc = lc, r.epi.ldd = N, r.epi.alpha = 1.f, r.epi.kind = E_NONE, r.epi.out_type = a.out_type;
            return launched(launch_reduce(r, st));
        }
        return DG_OK;
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_gemm_fp8");
    }
}

dg_status dg_gemm_fp8_grouped(dg_handle_t h, int64_t rows, int64_t N, int64_t K, int64_t experts, const void *A,
                              int64_t lda, const float *a_scale, int64_t lda_scale, const void *B, int64_t ldb,
                              int64_t stride_b, const float *b_scale, int64_t ldb_scale, int64_t stride_bs,
                              const int32_t *offsets, void *C, int32_t c_type, int64_t ldc, dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({rows, N, K, experts}));
        if (lda < 0 || ldb < 0 || lda_scale < 0 || ldb_scale < 0 || ldc < 0 || stride_b < 0 || stride_bs < 0)
            return api_fail(DG_ERR_INVALID_ARG, "negative size, stride or leading dimension");
        const int64_t la = lda ? lda : K, lb = ldb ? ldb : K, lc = ldc ? ldc : N, nsb = blocks_of(N);
        const int64_t lsa = lda_scale ? lda_scale : rows, lsb = ldb_scale ? ldb_scale : nsb;
        const int64_t xb = stride_b ? stride_b : N * lb, xs = stride_bs ? stride_bs : blocks_of(K) * lsb;
        if (la < K || lb < K || lc < N || lsa < rows || lsb < nsb)
            return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        if (rows == 0 || N == 0 || experts == 0) return DG_OK;
        if (!offsets) return api_fail(DG_ERR_INVALID_ARG, "offsets are required");
        Fp8Args a{};
        DG_TRY(check_out(C, c_type, a.out_type));
        if (K > 0) DG_TRY(check_operands(A, la, a_scale, B, lb, b_scale, K));
        if (K > 0 && xb % 16) return api_fail(DG_ERR_ALIGNMENT, "the experts' stride of B is a multiple of 16");
        if (!aligned(offsets, 4)) return api_fail(DG_ERR_ALIGNMENT, "offsets are 4-byte aligned");
        a.A = A, a.B = B, a.sa = a_scale, a.sb = b_scale, a.C = C, a.off = offsets;
        a.lda = la, a.ldb = lb, a.ld_sa = lsa, a.ld_sb = lsb, a.ldc = lc, a.stride_b = xb, a.stride_sb = xs;
        a.M = (int)rows, a.N = (int)N, a.K = (int)K, a.experts = (int)experts, a.split_k = 1;
        const bool exact = a.out_type == T_F32;
        return launched(launch_fp8(choose_rows(rows, experts, N, exact, huge_tile(exact, la, lb, K)), FP8_ROWS, FP8_BLOCK,
                                   a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_gemm_fp8_grouped");
    }
}

dg_status dg_gemm_fp8_wgrad(dg_handle_t h, int64_t M, int64_t N, int64_t rows, int64_t experts, const void *A,
                            int64_t lda, const float *a_scale, int64_t lda_scale, const void *B, int64_t ldb,
                            const float *b_scale, int64_t ldb_scale, const int32_t *offsets, void *C, int32_t c_type,
                            int64_t ldc, int64_t stride_c, dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({M, N, rows, experts}));
        if (lda < 0 || ldb < 0 || lda_scale < 0 || ldb_scale < 0 || ldc < 0 || stride_c < 0)
            return api_fail(DG_ERR_INVALID_ARG, "negative size, stride or leading dimension");
        const int64_t la = lda ? lda : rows, lb = ldb ? ldb : rows, lc = ldc ? ldc : N;
        const int64_t lsa = lda_scale ? lda_scale : M, lsb = ldb_scale ? ldb_scale : N;
        const int64_t xc = stride_c ? stride_c : M * lc;
        if (la < rows || lb < rows || lc < N || lsa < M || lsb < N)
            return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        if (M == 0 || N == 0 || experts == 0) return DG_OK;
        if (!experts_disjoint(M, N, lc, xc, experts))
            return api_fail(DG_ERR_INVALID_ARG, "the experts' matrices of C share elements");
        if (!offsets) return api_fail(DG_ERR_INVALID_ARG, "offsets are required");
        Fp8Args a{};
        DG_TRY(check_out(C, c_type, a.out_type));
        if (rows > 0) DG_TRY(check_operands(A, la, a_scale, B, lb, b_scale, rows));
        if (!aligned(offsets, 4)) return api_fail(DG_ERR_ALIGNMENT, "offsets are 4-byte aligned");
        a.A = A, a.B = B, a.sa = a_scale, a.sb = b_scale, a.C = C, a.off = offsets;
        a.lda = la, a.ldb = lb, a.ld_sa = lsa, a.ld_sb = lsb, a.ldc = lc, a.stride_c = xc;
        a.M = (int)M, a.N = (int)N, a.K = (int)rows, a.experts = (int)experts, a.split_k = 1;
        return launched(launch_fp8(choose_wgrad(M, N, experts, huge_tile(a.out_type == T_F32, la, lb, rows)), FP8_WGRAD, 1,
                                   a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_gemm_fp8_wgrad");
    }
}

dg_status dg_moe_sort_workspace(dg_handle_t h, int64_t tokens, int64_t topk, int64_t experts, int64_t *bytes)
{
    try {
        if (!api_live(h)) return api_fail(DG_ERR_INVALID_STATE, "handle is NULL or destroyed");
        if (!bytes) return api_fail(DG_ERR_INVALID_ARG, "bytes is NULL");
        DG_TRY(sizes_ok({tokens, topk, experts}));
        DG_TRY(sizes_ok({tokens * topk}));
        if (experts > MOE_MAX_EXPERTS) return api_fail(DG_ERR_UNSUPPORTED, "more than 512 experts");
        int blocks, per_block;
        moe_sort_shape(tokens * topk, blocks, per_block);
        *bytes = blocks > 1 ? (int64_t)blocks * experts * 4 : 0;
        return DG_OK;
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_moe_sort_workspace");
    }
}

dg_status dg_moe_sort(dg_handle_t h, int64_t tokens, int64_t topk, int64_t experts, int64_t align, const int32_t *ids,
                      int64_t capacity, int32_t *offsets, int32_t *src, int32_t *dst, void *workspace,
                      size_t workspace_bytes, dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({tokens, topk, experts, align, capacity}));
        DG_TRY(sizes_ok({tokens * topk}));
        if (experts < 1 || align < 1) return api_fail(DG_ERR_INVALID_ARG, "experts and align must be positive");
        if (experts > MOE_MAX_EXPERTS) return api_fail(DG_ERR_UNSUPPORTED, "more than 512 experts");
        const int64_t pairs = tokens * topk;
        // every expert that has a pair may round up
        if (pairs + std::min(pairs, experts) * (align - 1) > FP8_MOST)
            return api_fail(DG_ERR_UNSUPPORTED, "sizes above 2^31-4096 are not supported");
        if (capacity < pairs + std::min(pairs, experts) * (align - 1))
            return api_fail(DG_ERR_INVALID_ARG, "capacity does not hold every expert's rows rounded up to align");
        if (!offsets || (pairs > 0 && (!ids || !dst)) || (capacity > 0 && !src))
            return api_fail(DG_ERR_INVALID_ARG, "ids, offsets, src and dst are required");
        if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(src, 4) || !aligned(dst, 4))
            return api_fail(DG_ERR_ALIGNMENT, "index arrays are 4-byte aligned");
        MoeSortArgs a{};
        moe_sort_shape(pairs, a.blocks, a.per_block);
        if (a.blocks > 1) {
            const size_t need = (size_t)a.blocks * experts * 4;
            if (!workspace || workspace_bytes < need)
                return api_fail(DG_ERR_WORKSPACE, "workspace missing or smaller than " + std::to_string(need) + " bytes");
            if (!aligned(workspace, 4)) return api_fail(DG_ERR_ALIGNMENT, "workspace must be 4-byte aligned");
        }
        a.ids = ids, a.off = offsets, a.src = src, a.dst = dst, a.ws = reinterpret_cast<int32_t *>(workspace);
        a.pairs = (int)pairs, a.experts = (int)experts, a.align = (int)align, a.capacity = (int)capacity;
        return launched(launch_moe_sort(a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_moe_sort");
    }
}

dg_status dg_moe_gather(dg_handle_t h, int64_t rows, int64_t hidden, const void *X, int32_t type, int64_t tokens,
                        int64_t ldx, const int32_t *src, int64_t topk, void *Y, int64_t ldy, dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({rows, hidden, tokens, topk}));
        const int elt = elt_of(type);
        if (elt < 0) return api_fail(DG_ERR_UNSUPPORTED, "rows are F16, BF16 or F32");
        const int64_t lx = ldx ? ldx : hidden, ly = ldy ? ldy : hidden;
        if (topk < 1) return api_fail(DG_ERR_INVALID_ARG, "topk must be positive");
        if (lx < hidden || ly < hidden) return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        if (rows == 0 || hidden == 0) return DG_OK;
        if ((!X && tokens > 0) || !src || !Y) return api_fail(DG_ERR_INVALID_ARG, "X, src and Y are required");
        if (!aligned(X, elt_bytes(elt)) || !aligned(Y, elt_bytes(elt)) || !aligned(src, 4))
            return api_fail(DG_ERR_ALIGNMENT, "a pointer is misaligned for its type");
        MoeMoveArgs a{};
        a.x = X, a.out = Y, a.src = src, a.ldx = lx, a.ldout = ly;
        a.rows = (int)rows, a.tokens = (int)tokens, a.topk = (int)topk, a.hidden = (int)hidden, a.type = elt;
        return launched(launch_moe_gather(a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_moe_gather");
    }
}

dg_status dg_moe_combine(dg_handle_t h, int64_t tokens, int64_t topk, int64_t hidden, const void *Y, int32_t type,
                         int64_t rows, int64_t ldy, const int32_t *dst, const float *weights, void *O, int64_t ldo,
                         dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({tokens, topk, hidden, rows}));
        DG_TRY(sizes_ok({tokens * topk}));
        const int elt = elt_of(type);
        if (elt < 0) return api_fail(DG_ERR_UNSUPPORTED, "rows are F16, BF16 or F32");
        const int64_t ly = ldy ? ldy : hidden, lo = ldo ? ldo : hidden;
        if (ly < hidden || lo < hidden) return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        if (tokens == 0 || hidden == 0) return DG_OK;
        if ((!Y && rows > 0) || (!dst && topk > 0) || !O) return api_fail(DG_ERR_INVALID_ARG, "Y, dst and O are required");
        if (!aligned(Y, elt_bytes(elt)) || !aligned(O, elt_bytes(elt)) || !aligned(dst, 4) || !aligned(weights, 4))
            return api_fail(DG_ERR_ALIGNMENT, "a pointer is misaligned for its type");
        MoeMoveArgs a{};
        a.x = Y, a.out = O, a.dst = dst, a.w = weights, a.ldx = ly, a.ldout = lo;
        a.rows = (int)rows, a.tokens = (int)tokens, a.topk = (int)topk, a.hidden = (int)hidden, a.type = elt;
        return launched(launch_moe_combine(a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_moe_combine");
    }
}

dg_status dg_moe_combine_grad(dg_handle_t h, int64_t tokens, int64_t topk, int64_t hidden, int64_t rows,
                              const void *dO, int32_t type, int64_t lddo, const void *Y, int64_t ldy,
                              const int32_t *dst, const int32_t *src, const float *weights, void *dY, int64_t lddy,
                              float *dW, dg_stream_t stream)
{
    try {
        DG_TRY(device_ready(h));
        DG_TRY(sizes_ok({tokens, topk, hidden, rows}));
        DG_TRY(sizes_ok({tokens * topk}));
        const int elt = elt_of(type);
        if (elt < 0) return api_fail(DG_ERR_UNSUPPORTED, "rows are F16, BF16 or F32");
        const int64_t ld = lddo ? lddo : hidden, ly = ldy ? ldy : hidden, lg = lddy ? lddy : hidden;
        if (ld < hidden || ly < hidden || lg < hidden)
            return api_fail(DG_ERR_INVALID_ARG, "a leading dimension is smaller than the matrix");
        const int64_t pairs = tokens * topk;
        if (pairs == 0 && rows == 0) return DG_OK;
        if ((pairs > 0 && (!dst || (!dO && hidden > 0))) || (rows > 0 && (!src || (!dY && hidden > 0))))
            return api_fail(DG_ERR_INVALID_ARG, "dO, dst, src and dY are required");
        if (dW && !Y && rows > 0 && hidden > 0) return api_fail(DG_ERR_INVALID_ARG, "the weights' gradient needs Y");
        if (!aligned(dO, elt_bytes(elt)) || !aligned(Y, elt_bytes(elt)) || !aligned(dY, elt_bytes(elt)) ||
            !aligned(dst, 4) || !aligned(src, 4) || !aligned(weights, 4) || !aligned(dW, 4))
            return api_fail(DG_ERR_ALIGNMENT, "a pointer is misaligned for its type");
        MoeMoveArgs a{};
        a.x = Y, a.dout = dO, a.out = dY, a.src = src, a.dst = dst, a.w = weights, a.dw = dW;
        a.ldx = ly, a.ldout = lg, a.ld_dout = ld;
        a.rows = (int)rows, a.tokens = (int)tokens, a.topk = (int)topk, a.hidden = (int)hidden, a.type = elt;
        return launched(launch_moe_combine_grad(a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return api_fail(DG_ERR_INTERNAL, "exception in dg_moe_combine_grad");
    }
}

}  // extern "C"
