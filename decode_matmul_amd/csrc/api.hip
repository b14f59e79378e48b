// extern "C" entry points: argument validation on the host, then launches on
// the caller's stream.  No memory is allocated and no state is kept.
#include <stddef.h>

#include "common.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool group_ok(int G) { return G == 64 || G == 128; }

int hip_status(hipError_t e) { return e == hipSuccess ? TQ_OK : TQ_ERR_HIP; }

// Launchers that refuse too large a grid themselves say so with hipErrorInvalidConfiguration.
int grid_status(hipError_t e) { return e == hipErrorInvalidConfiguration ? TQ_ERR_SHAPE : hip_status(e); }

bool is_dtype(int32_t d) { return d == TQ_F32 || d == TQ_BF16; }

uintptr_t bytes_of(int32_t d) { return d == TQ_F32 ? 4 : 2; }

// Rows of `cols` elements, `ld` apart (one row has no distance).
bool rows_ok(int64_t rows, int64_t cols, int64_t ld) { return rows <= 1 || (ld >= cols && ld < kMaxDim); }

}  // namespace

extern "C" {

const char* tq_status_string(int status) {
    switch (status) {
        case TQ_OK: return "ok";
        case TQ_ERR_NULL: return "a required pointer is NULL";
        case TQ_ERR_SHAPE: return "a size is negative, inconsistent or too large";
        case TQ_ERR_UNSUPPORTED: return "unsupported group size, plane count or mode";
        case TQ_ERR_DTYPE: return "unknown dtype";
        case TQ_ERR_ALIGN: return "a pointer is not aligned as documented";
        case TQ_ERR_HIP: return "the HIP runtime rejected a launch";
        case TQ_ERR_SCRATCH:
            return "the call needs more device scratch than DMM_SCRATCH_BYTES (34 MiB)";
        default: return "unknown status";
    }
}

int tq_pack(const float* W, int64_t rows, int64_t K, int32_t G, int32_t planes,
            uint8_t* codes1, uint16_t* scales1, uint8_t* codes2, uint16_t* scales2,
            int32_t* d_status, void* stream) {
    if (!W || !codes1 || !scales1 || !d_status) return TQ_ERR_NULL;
    if (rows < 0 || K < 0 || rows >= kMaxDim || K >= kMaxDim) return TQ_ERR_SHAPE;
    if (!group_ok(G) || (planes != 1 && planes != 2)) return TQ_ERR_UNSUPPORTED;
    if (planes == 2 && (!codes2 || !scales2)) return TQ_ERR_NULL;
    if (planes == 1 && (codes2 || scales2)) return TQ_ERR_SHAPE;
    if (!aligned(W, 4) || !aligned(scales1, 2) || (scales2 && !aligned(scales2, 2)) ||
        !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    const int64_t groups = rows * ((K + G - 1) / G);
    if (groups / 128 >= kMaxDim) return TQ_ERR_SHAPE;   // grid: 128 or 256 groups a workgroup
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = dmm::launch_status_clear(d_status, s);
    if (e != hipSuccess) return TQ_ERR_HIP;
    return hip_status(dmm::launch_pack(W, rows, K, G, planes, codes1, scales1, codes2, scales2,
                                       d_status, s));
}

int rb_encode(const float* W, int64_t N, int64_t K, const float* ladder, float zeta,
              int32_t rho_rows, uint8_t* codes, float* alpha_out, uint16_t* row_scale,
              int32_t* d_status, void* stream) {
    if (!ladder || !alpha_out || !d_status) return TQ_ERR_NULL;
    if (N < 0 || K < 0 || N >= kMaxDim || K >= kMaxDim) return TQ_ERR_SHAPE;
    if (rho_rows < 0) return TQ_ERR_SHAPE;
    if (!(zeta >= 0.f && zeta <= 1.f)) return TQ_ERR_UNSUPPORTED;
    for (int i = 0; i < 5; ++i)                       // finite, nonnegative steps
        if (!(ladder[i] >= 0.f && ladder[i] <= 3.402823466e38f)) return TQ_ERR_UNSUPPORTED;
    if (N > 0 && K > 0 && (!W || !codes)) return TQ_ERR_NULL;
    if (rho_rows > 0 && N > 0 && !row_scale) return TQ_ERR_NULL;
    if (rho_rows == 0 && row_scale) return TQ_ERR_SHAPE;
    if ((W && !aligned(W, 4)) || !aligned(alpha_out, 4) || (row_scale && !aligned(row_scale, 2)) ||
        !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    return hip_status(dmm::launch_rb_encode(W, N, K, ladder, zeta, rho_rows, codes, alpha_out,
                                            row_scale, d_status, (hipStream_t)stream));
}

int tq_unpack(const uint8_t* codes, const uint16_t* scales, int64_t rows, int64_t K,
              int32_t G, void* W_out, int32_t out_dtype, int32_t* d_status, void* stream) {
    if (!codes || !scales || !W_out || !d_status) return TQ_ERR_NULL;
    if (rows < 0 || K < 0 || rows >= kMaxDim || K >= kMaxDim) return TQ_ERR_SHAPE;
    if (!group_ok(G)) return TQ_ERR_UNSUPPORTED;
    if (out_dtype != TQ_F32 && out_dtype != TQ_BF16) return TQ_ERR_DTYPE;
    if (!aligned(scales, 2) || !aligned(W_out, out_dtype == TQ_F32 ? 4 : 2) ||
        !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    const int64_t groups = rows * ((K + G - 1) / G);
    if (groups / 128 >= kMaxDim) return TQ_ERR_SHAPE;   // grid: 128 or 256 groups a workgroup
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = dmm::launch_status_clear(d_status, s);
    if (e != hipSuccess) return TQ_ERR_HIP;
    return hip_status(dmm::launch_unpack(codes, scales, rows, K, G, W_out, out_dtype, d_status, s));
}

// tq_matmul and tq_matmul_hot: n_hot < 0 gives every expert the planes
// passed; 0 <= n_hot <= n_experts gives plane 2 to experts 0 .. n_hot - 1.
static int tq_matmul_common(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes1,
                            const uint16_t* scales1, const uint8_t* codes2,
                            const uint16_t* scales2, int32_t n_hot, int64_t N, int32_t G,
                            int32_t n_experts, const int32_t* expert_ids, int32_t top_k, void* y,
                            int32_t y_dtype, void* stream, void* workspace = nullptr,
                            int64_t workspace_bytes = 0) {
    if (M < 0 || K < 0 || N < 0 || M >= kMaxDim || K >= kMaxDim || N >= kMaxDim)
        return TQ_ERR_SHAPE;
    if (!group_ok(G)) return TQ_ERR_UNSUPPORTED;
    if (K % G != 0) return TQ_ERR_SHAPE;
    if (y_dtype != TQ_F32 && y_dtype != TQ_BF16) return TQ_ERR_DTYPE;
    if (n_experts < 0) return TQ_ERR_SHAPE;
    if ((codes2 == nullptr) != (scales2 == nullptr)) return TQ_ERR_NULL;
    if (n_experts > 0) {
        if (top_k < 1) return TQ_ERR_SHAPE;
        if (M * (int64_t)top_k > dmm::tq_max_grouped_pairs()) return TQ_ERR_SHAPE;
    }
    if (M == 0 || N == 0) return TQ_OK;
    if (!y || (K > 0 && (!x || !codes1 || !scales1))) return TQ_ERR_NULL;
    if (n_experts > 0 && !expert_ids) return TQ_ERR_NULL;
    if (!aligned(x, 2) || !aligned(scales1, 2) || (scales2 && !aligned(scales2, 2)) ||
        !aligned(y, y_dtype == TQ_F32 ? 4 : 2) || (expert_ids && !aligned(expert_ids, 4)))
        return TQ_ERR_ALIGN;
    const int64_t row_blocks = (N + 15) / 16;
    if (row_blocks * (n_experts > 0 ? n_experts : 1) >= kMaxDim) return TQ_ERR_SHAPE;
    dmm::TqMatmulArgs a;
    a.x = x;
    a.M = M;
    a.K = K;
    a.N = N;
    a.codes[0] = codes1;
    a.codes[1] = codes2;
    a.scales[0] = scales1;
    a.scales[1] = scales2;
    a.planes = codes2 ? 2 : 1;
    a.G = G;
    a.n_experts = n_experts;
    a.ids = n_experts > 0 ? expert_ids : nullptr;
    a.top_k = n_experts > 0 ? top_k : 1;
    a.y = y;
    a.y_dtype = y_dtype;
    a.e_begin = 0;
    a.e_end = n_experts;
    a.nan_rows = true;
    a.workspace = nullptr;
    if (workspace) {
        if (!aligned(workspace, 256)) return TQ_ERR_ALIGN;
        if (workspace_bytes < dmm::tq_prefill_ws_bytes(M, K)) return TQ_ERR_SHAPE;
        a.workspace = workspace;
    }
    hipStream_t s = (hipStream_t)stream;
    if (n_hot < 0 || n_hot == n_experts) return hip_status(dmm::launch_tq_matmul(a, s));
    if (n_hot == 0) {
        a.planes = 1;
        a.codes[1] = nullptr;
        a.scales[1] = nullptr;
        return hip_status(dmm::launch_tq_matmul(a, s));
    }
    // hot prefix: experts 0 .. n_hot - 1 with both planes, the rest with one
    // (disjoint output slots; the cold launch writes the rows of invalid ids)
    dmm::TqMatmulArgs hot = a;
    hot.e_end = n_hot;
    hot.nan_rows = false;
    dmm::TqMatmulArgs cold = a;
    cold.planes = 1;
    cold.codes[1] = nullptr;
    cold.scales[1] = nullptr;
    cold.e_begin = n_hot;
    hipError_t e = hipSuccess;
    if (dmm::launch_tq_wave_hot(hot, cold, s, &e)) return hip_status(e);   // one launch
    if (dmm::launch_tq_rows_hot(hot, cold, s, &e)) return hip_status(e);
    e = dmm::launch_tq_matmul(hot, s);
    if (e != hipSuccess) return TQ_ERR_HIP;
    return hip_status(dmm::launch_tq_matmul(cold, s));
}

int tq_matmul(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes1,
              const uint16_t* scales1, const uint8_t* codes2, const uint16_t* scales2,
              int64_t N, int32_t G, int32_t n_experts, const int32_t* expert_ids,
              int32_t top_k, void* y, int32_t y_dtype, void* stream) {
    return tq_matmul_common(x, M, K, codes1, scales1, codes2, scales2, -1, N, G, n_experts,
                            expert_ids, top_k, y, y_dtype, stream);
}

int64_t tq_prefill_workspace_bytes(int64_t M, int64_t K) {
    if (M < 0 || K < 0 || M >= kMaxDim || K >= kMaxDim) return -1;
    return dmm::tq_prefill_ws_bytes(M, K);
}

int tq_matmul_ws(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes1,
                 const uint16_t* scales1, const uint8_t* codes2, const uint16_t* scales2,
                 int64_t N, int32_t G, void* y, int32_t y_dtype, void* workspace,
                 int64_t workspace_bytes, void* stream) {
    return tq_matmul_common(x, M, K, codes1, scales1, codes2, scales2, -1, N, G, 0, nullptr, 1, y,
                            y_dtype, stream, workspace, workspace_bytes);
}

int tq_matmul_hot(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes1,
                  const uint16_t* scales1, const uint8_t* codes2, const uint16_t* scales2,
                  int32_t n_hot, int64_t N, int32_t G, int32_t n_experts,
                  const int32_t* expert_ids, int32_t top_k, void* y, int32_t y_dtype,
                  void* stream) {
    if (n_experts < 1) return TQ_ERR_UNSUPPORTED;     // grouped calls only
    if (n_hot < 0 || n_hot > n_experts) return TQ_ERR_SHAPE;
    if (n_hot > 0 && (!codes2 || !scales2)) return TQ_ERR_NULL;
    if (n_hot == 0 && (codes2 || scales2)) return TQ_ERR_SHAPE;
    return tq_matmul_common(x, M, K, codes1, scales1, codes2, scales2, n_hot, N, G, n_experts,
                            expert_ids, top_k, y, y_dtype, stream);
}

int rb_table(const float* ladder, float* table_out) {
    if (!ladder || !table_out) return TQ_ERR_NULL;
    for (int b = 0; b < 243; ++b) {
        double acc = 0.0;
        int p3 = 81;                               // 3^(5-i) for i = 1
        for (int i = 0; i < 5; ++i) {
            const int c = (b / p3) % 3 - 1;        // c_1 is the most significant digit
            acc += (double)c * (double)ladder[i];
            p3 /= 3;
        }
        table_out[b] = (float)acc;                 // one nearest-even rounding
    }
    return TQ_OK;
}

int rb_matmul(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes, int64_t N,
              const float* table, float alpha, const uint16_t* row_scale, const float* bias,
              void* y, int32_t y_dtype, void* stream) {
    return rb_matmul_rho_block(x, M, K, codes, N, table, alpha, row_scale, 1, bias, y, y_dtype,
                               stream);
}

// Every Route B matmul: code bytes (used == NULL) or 7-bit indices, one code
// book (table_rows == 0) or one per block of table_rows rows.
static int rb_matmul_common(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes,
                            const uint8_t* used, int64_t N, const float* table,
                            int32_t table_rows, float alpha, const uint16_t* row_scale,
                            int32_t rho_rows, const float* bias, void* y, int32_t y_dtype,
                            void* stream, void* workspace = nullptr, int64_t workspace_bytes = 0,
                            bool static_scratch = false) {
    if (M < 0 || K < 0 || N < 0 || M >= kMaxDim || K >= kMaxDim || N >= kMaxDim)
        return TQ_ERR_SHAPE;
    if (rho_rows < 1 || table_rows < 0) return TQ_ERR_SHAPE;
    if (table_rows % 32 != 0) return TQ_ERR_UNSUPPORTED;
    if (y_dtype != TQ_F32 && y_dtype != TQ_BF16) return TQ_ERR_DTYPE;
    if (M == 0 || N == 0) return TQ_OK;
    if (!table || !y || (K > 0 && (!x || !codes))) return TQ_ERR_NULL;
    if (!aligned(x, 2) || !aligned(table, 4) || (row_scale && !aligned(row_scale, 2)) ||
        (bias && !aligned(bias, 4)) || !aligned(y, y_dtype == TQ_F32 ? 4 : 2))
        return TQ_ERR_ALIGN;
    dmm::RbMatmulArgs a;
    a.x = x;
    a.M = M;
    a.K = K;
    a.N = N;
    a.codes = codes;
    a.used = used;
    a.table = table;
    a.table_rows = table_rows;
    a.alpha = alpha;
    a.row_scale = row_scale;
    a.rho_rows = rho_rows;
    a.bias = bias;
    a.y = y;
    a.y_dtype = y_dtype;
    a.workspace = nullptr;
    hipStream_t s = (hipStream_t)stream;
    if (M <= 16) {
        if ((N + 15) / 16 >= kMaxDim) return TQ_ERR_SHAPE;
        return hip_status(used ? dmm::launch_rb7_gemv(a, s) : dmm::launch_rb_gemv(a, s));
    }
    if ((M + 255) / 256 >= 65536) return TQ_ERR_SHAPE;
    if (static_scratch) {
        // the library's own per-device array stands in for the workspace
        if (dmm::rb_prefill_ws_bytes(M, K) > dmm::kScratchBytes) return TQ_ERR_SCRATCH;
        if (dmm::scratch_of_current_device(&workspace) != hipSuccess) return TQ_ERR_HIP;
        workspace_bytes = dmm::kScratchBytes;
    }
    if (workspace) {
        if (!aligned(workspace, 256)) return TQ_ERR_ALIGN;
        if (workspace_bytes < dmm::rb_prefill_ws_bytes(M, K)) return TQ_ERR_SHAPE;
        a.workspace = workspace;
    }
    return hip_status(dmm::launch_rb_prefill(a, s));
}

int64_t rb_prefill_workspace_bytes(int64_t M, int64_t K) {
    if (M < 0 || K < 0 || M >= kMaxDim || K >= kMaxDim) return -1;
    return dmm::rb_prefill_ws_bytes(M, K);
}

int rb_matmul_ws(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes, int64_t N,
                 const float* tables, int32_t table_rows, float alpha, const uint16_t* row_scale,
                 int32_t rho_rows, const float* bias, void* y, int32_t y_dtype, void* workspace,
                 int64_t workspace_bytes, void* stream) {
    return rb_matmul_common(x, M, K, codes, nullptr, N, tables, table_rows, alpha, row_scale,
                            rho_rows, bias, y, y_dtype, stream, workspace, workspace_bytes);
}

int rb_matmul_noalloc(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes, int64_t N,
                      const float* tables, int32_t table_rows, float alpha,
                      const uint16_t* row_scale, int32_t rho_rows, const float* bias, void* y,
                      int32_t y_dtype, void* stream) {
    return rb_matmul_common(x, M, K, codes, nullptr, N, tables, table_rows, alpha, row_scale,
                            rho_rows, bias, y, y_dtype, stream, nullptr, 0, true);
}

int rb_matmul_rho_block(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes, int64_t N,
                        const float* table, float alpha, const uint16_t* row_scale,
                        int32_t rho_rows, const float* bias, void* y, int32_t y_dtype,
                        void* stream) {
    return rb_matmul_common(x, M, K, codes, nullptr, N, table, 0, alpha, row_scale, rho_rows,
                            bias, y, y_dtype, stream);
}

int rb_matmul_blocks(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes, int64_t N,
                     const float* tables, int32_t table_rows, float alpha,
                     const uint16_t* row_scale, int32_t rho_rows, const float* bias, void* y,
                     int32_t y_dtype, void* stream) {
    return rb_matmul_common(x, M, K, codes, nullptr, N, tables, table_rows, alpha, row_scale,
                            rho_rows, bias, y, y_dtype, stream);
}

int rb_truncate(const uint8_t* codes, int64_t N, int64_t K, uint8_t* used_out,
                int32_t* n_used_out, uint8_t* codes7, int32_t* d_status, void* stream) {
    if (!used_out || !n_used_out || !d_status) return TQ_ERR_NULL;
    if (N < 0 || K < 0 || N >= kMaxDim || K >= kMaxDim) return TQ_ERR_SHAPE;
    if (N > 0 && K > 0 && (!codes || !codes7)) return TQ_ERR_NULL;
    if (!aligned(used_out, 4) || !aligned(n_used_out, 4) || !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    return hip_status(dmm::launch_rb_truncate(codes, N, K, used_out, n_used_out, codes7, d_status,
                                              (hipStream_t)stream));
}

int rb_matmul7(const uint16_t* x, int64_t M, int64_t K, const uint8_t* codes7, int64_t N,
               const uint8_t* used, const float* tables, int32_t table_rows, float alpha,
               const uint16_t* row_scale, int32_t rho_rows, const float* bias, void* y,
               int32_t y_dtype, void* stream) {
    if (!used) return TQ_ERR_NULL;
    return rb_matmul_common(x, M, K, codes7, used, N, tables, table_rows, alpha, row_scale,
                            rho_rows, bias, y, y_dtype, stream);
}

int mx_pack(const void* W, int32_t w_dtype, int64_t rows, int64_t K, int64_t ldw, uint8_t* codes,
            uint8_t* scales, int32_t* d_status, void* stream) {
    if (rows < 0 || K < 0 || rows >= kMaxDim || K >= kMaxDim || !rows_ok(rows, K, ldw)) return TQ_ERR_SHAPE;
    if (!is_dtype(w_dtype)) return TQ_ERR_DTYPE;
    if (rows > 0 && K > 0 && (!W || !codes || !scales)) return TQ_ERR_NULL;
    if (!aligned(W, bytes_of(w_dtype)) || !aligned(codes, 16) || !aligned(d_status, 4)) return TQ_ERR_ALIGN;
    if (!dmm::grid_fits(rows * ((K + 31) / 32) / 64 + 1, 256)) return TQ_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    if (d_status && dmm::launch_status_clear(d_status, s) != hipSuccess) return TQ_ERR_HIP;
    return grid_status(dmm::launch_mx_pack(W, w_dtype, rows, K, ldw, codes, scales, d_status, s));
}

int mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* W_out,
              int32_t out_dtype, int32_t* d_status, void* stream) {
    if (rows < 0 || K < 0 || rows >= kMaxDim || K >= kMaxDim) return TQ_ERR_SHAPE;
    if (!is_dtype(out_dtype)) return TQ_ERR_DTYPE;
    if (rows > 0 && K > 0 && (!W_out || !codes || !scales)) return TQ_ERR_NULL;
    if (!aligned(W_out, bytes_of(out_dtype)) || !aligned(codes, 16) || !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    if (!dmm::grid_fits(rows * ((K + 31) / 32) / 32 + 1, 256)) return TQ_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    if (d_status && dmm::launch_status_clear(d_status, s) != hipSuccess) return TQ_ERR_HIP;
    return grid_status(dmm::launch_mx_unpack(codes, scales, rows, K, W_out, out_dtype, d_status, s));
}

// Every MXFP4 product; a holds the call's arguments, x_any its activations.
static int mx_matmul_common(dmm::MxMatmulArgs& a, const void* x_any, bool x_rows_ok, void* stream) {
    if (a.M < 0 || a.K < 0 || a.N < 0 || a.M >= kMaxDim || a.K >= dmm::kMxMaxK || a.N >= kMaxDim || !x_rows_ok)
        return TQ_ERR_SHAPE;
    if (!is_dtype(a.y_dtype)) return TQ_ERR_DTYPE;
    if (a.M == 0 || a.N == 0) return TQ_OK;
    if (!a.y || (a.K > 0 && (!x_any || !a.codes || !a.scales))) return TQ_ERR_NULL;
    if (!aligned(a.x, 2) || !aligned(a.x_codes, 16) || !aligned(a.codes, 16) || !aligned(a.bias, 4) ||
        !aligned(a.y, bytes_of(a.y_dtype)))
        return TQ_ERR_ALIGN;
    return grid_status(dmm::launch_mx_matmul(a, (hipStream_t)stream));
}

int mx_matmul(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* codes,
              const uint8_t* scales, int64_t N, const float* bias, void* y, int32_t y_dtype,
              void* stream) {
    dmm::MxMatmulArgs a = {x,    ldx, nullptr, nullptr, M, K, N,      codes, scales,
                           bias, 0,   nullptr, nullptr, 1, y, y_dtype};
    return mx_matmul_common(a, x, rows_ok(M, K, ldx), stream);
}

int mx_matmul_mx(const uint8_t* x_codes, const uint8_t* x_scales, int64_t M, int64_t K,
                 const uint8_t* codes, const uint8_t* scales, int64_t N, const float* bias, void* y,
                 int32_t y_dtype, void* stream) {
    dmm::MxMatmulArgs a = {nullptr, 0, x_codes, x_scales, M, K, N,      codes, scales,
                           bias,    0, nullptr, nullptr,  1, y, y_dtype};
    return mx_matmul_common(a, x_codes && x_scales ? x_codes : nullptr, true, stream);
}

int mx_matmul_experts(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* codes,
                      const uint8_t* scales, int64_t N, int32_t n_experts, const float* bias,
                      const int32_t* offsets, const int32_t* order, int32_t top_k, void* y,
                      int32_t y_dtype, void* stream) {
    if (n_experts < 1 || top_k < 1) return TQ_ERR_SHAPE;
    if (M >= 0 && M < kMaxDim && M * top_k >= kMaxDim) return TQ_ERR_SHAPE;
    if (M > 0 && N > 0 && (!offsets || !order)) return TQ_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(order, 4)) return TQ_ERR_ALIGN;
    dmm::MxMatmulArgs a = {x,    ldx,       nullptr, nullptr, M,     K, N,      codes, scales,
                           bias, n_experts, offsets, order,   top_k, y, y_dtype};
    return mx_matmul_common(a, x, rows_ok(M, K, ldx), stream);
}

int64_t moe_route_workspace_bytes(int64_t M, int32_t top_k, int32_t n_experts) {
    if (M < 0 || M >= kMaxDim || top_k < 1 || M * top_k >= kMaxDim || n_experts < 1 ||
        n_experts > dmm::kMoeMaxExperts)
        return -1;
    return dmm::moe_route_ws_bytes(M * top_k, n_experts);
}

int moe_route(const int32_t* expert_ids, int64_t M, int32_t top_k, int32_t n_experts,
              int32_t* counts, int32_t* offsets, int32_t* order, void* workspace,
              int64_t workspace_bytes, void* stream) {
    if (n_experts > dmm::kMoeMaxExperts) return TQ_ERR_UNSUPPORTED;
    const int64_t need = moe_route_workspace_bytes(M, top_k, n_experts);
    if (need < 0) return TQ_ERR_SHAPE;
    if (!counts || !offsets || (M > 0 && (!expert_ids || !order))) return TQ_ERR_NULL;
    if (need > 0 && !workspace) return TQ_ERR_NULL;
    if (!aligned(expert_ids, 4) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(order, 4) ||
        !aligned(workspace, 4))
        return TQ_ERR_ALIGN;
    if (need > 0 && workspace_bytes < need) return TQ_ERR_SHAPE;
    return hip_status(dmm::launch_moe_route(expert_ids, M * top_k, n_experts, counts, offsets, order,
                                            workspace, (hipStream_t)stream));
}

int64_t moe_balance_workspace_bytes(int64_t M, int32_t n_experts) {
    if (M < 0 || M >= kMaxDim || n_experts < 1 || n_experts > dmm::kMoeMaxExperts) return -1;
    return dmm::moe_balance_ws_bytes(M, n_experts);
}

int moe_balance(const void* logits, int32_t l_dtype, int64_t M, int32_t n_experts, int64_t ldl,
                const uint8_t* token_mask, const int32_t* counts, float* loss, float* weights,
                void* workspace, int64_t workspace_bytes, void* stream) {
    if (n_experts > dmm::kMoeMaxExperts) return TQ_ERR_UNSUPPORTED;
    const int64_t need = moe_balance_workspace_bytes(M, n_experts);
    if (need < 0 || !rows_ok(M, n_experts, ldl)) return TQ_ERR_SHAPE;
    if (!is_dtype(l_dtype)) return TQ_ERR_DTYPE;
    if (!counts || !loss || !weights || (M > 0 && !logits) || (need > 0 && !workspace)) return TQ_ERR_NULL;
    if (!aligned(logits, bytes_of(l_dtype)) || !aligned(counts, 4) || !aligned(loss, 4) ||
        !aligned(weights, 4) || !aligned(workspace, 8))
        return TQ_ERR_ALIGN;
    if (need > 0 && workspace_bytes < need) return TQ_ERR_SHAPE;
    return hip_status(dmm::launch_moe_balance(logits, l_dtype, M, n_experts, ldl, token_mask, counts, loss,
                                              weights, workspace, (hipStream_t)stream));
}

int moe_balance_grad(const void* logits, int32_t l_dtype, int64_t M, int32_t n_experts, int64_t ldl,
                     const uint8_t* token_mask, const float* weights, const float* dloss,
                     void* dlogits, void* stream) {
    if (n_experts > dmm::kMoeMaxExperts) return TQ_ERR_UNSUPPORTED;
    if (M < 0 || M >= kMaxDim || n_experts < 1 || !rows_ok(M, n_experts, ldl)) return TQ_ERR_SHAPE;
    if (!is_dtype(l_dtype)) return TQ_ERR_DTYPE;
    if (M == 0) return TQ_OK;
    if (!logits || !weights || !dloss || !dlogits) return TQ_ERR_NULL;
    if (!aligned(logits, bytes_of(l_dtype)) || !aligned(weights, 4) || !aligned(dloss, 4) ||
        !aligned(dlogits, bytes_of(l_dtype)))
        return TQ_ERR_ALIGN;
    return grid_status(dmm::launch_moe_balance_grad(logits, l_dtype, M, n_experts, ldl, token_mask, weights,
                                                    dloss, dlogits, (hipStream_t)stream));
}

// --------------------------------------------------- e4m3 blocks of 128

int f8_pack(const void* W, int32_t w_dtype, int64_t rows, int64_t K, int64_t ldw, int32_t block_rows,
            uint8_t* codes, float* scales, int32_t* d_status, void* stream) {
    if (block_rows != 1 && block_rows != 128) return TQ_ERR_UNSUPPORTED;
    if (rows < 0 || K < 0 || rows >= kMaxDim || K >= dmm::kMxMaxK || !rows_ok(rows, K, ldw)) return TQ_ERR_SHAPE;
    if (!is_dtype(w_dtype)) return TQ_ERR_DTYPE;
    if (rows > 0 && K > 0 && (!W || !codes || !scales)) return TQ_ERR_NULL;
    if (!aligned(W, bytes_of(w_dtype)) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    if (!dmm::grid_fits(rows * ((K + 127) / 128) / 16 + 1, 256)) return TQ_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    if (d_status && dmm::launch_status_clear(d_status, s) != hipSuccess) return TQ_ERR_HIP;
    return grid_status(dmm::launch_f8_pack(W, w_dtype, rows, K, ldw, block_rows, codes, scales, d_status, s));
}

int f8_unpack(const uint8_t* codes, const float* scales, int64_t rows, int64_t K, int32_t block_rows,
              void* W_out, int32_t out_dtype, int32_t* d_status, void* stream) {
    if (block_rows != 1 && block_rows != 128) return TQ_ERR_UNSUPPORTED;
    if (rows < 0 || K < 0 || rows >= kMaxDim || K >= dmm::kMxMaxK) return TQ_ERR_SHAPE;
    if (!is_dtype(out_dtype)) return TQ_ERR_DTYPE;
    if (rows > 0 && K > 0 && (!W_out || !codes || !scales)) return TQ_ERR_NULL;
    if (!aligned(W_out, bytes_of(out_dtype)) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    if (!dmm::grid_fits(rows * ((K + 127) / 128) / 16 + 1, 256)) return TQ_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    if (d_status && dmm::launch_status_clear(d_status, s) != hipSuccess) return TQ_ERR_HIP;
    return grid_status(dmm::launch_f8_unpack(codes, scales, rows, K, block_rows, W_out, out_dtype, d_status, s));
}

int f8_norm_pack(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, const void* residual,
                 int64_t ldr, const void* weight, int32_t w_dtype, double eps, void* h_out, int64_t ldh,
                 void* y_out, int64_t ldy, uint8_t* codes, float* scales, int32_t* d_status, void* stream) {
    if (M < 0 || K < 0 || M >= kMaxDim || K >= dmm::kMxMaxK || !rows_ok(M, K, ldx) || !(eps >= 0.0) ||
        (residual && !rows_ok(M, K, ldr)) || (h_out && !rows_ok(M, K, ldh)) || (y_out && !rows_ok(M, K, ldy)))
        return TQ_ERR_SHAPE;
    if (!is_dtype(x_dtype) || !is_dtype(w_dtype)) return TQ_ERR_DTYPE;
    if (M > 0 && K > 0 && (!x || !weight || !codes || !scales)) return TQ_ERR_NULL;
    const uintptr_t xb = bytes_of(x_dtype);
    if (!aligned(x, xb) || !aligned(residual, xb) || !aligned(h_out, xb) || !aligned(y_out, xb) ||
        !aligned(weight, bytes_of(w_dtype)) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(d_status, 4))
        return TQ_ERR_ALIGN;
    if (!dmm::grid_fits(M, 1024)) return TQ_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    if (d_status && dmm::launch_status_clear(d_status, s) != hipSuccess) return TQ_ERR_HIP;
    const dmm::F8NormArgs a = {x,   x_dtype, M,   K,     ldx, residual, ldr,    weight, w_dtype,
                               eps, h_out,   ldh, y_out, ldy, codes,    scales, d_status};
    return grid_status(dmm::launch_f8_norm_pack(a, s));
}

// An e4m3 product takes DMM_SHORT_SUMS with TQ_BF16 only; any other type with it is none.
static bool short_sums(int32_t y_dtype) { return y_dtype == (TQ_BF16 | DMM_SHORT_SUMS); }
static int32_t plain(int32_t y_dtype) { return short_sums(y_dtype) ? TQ_BF16 : y_dtype; }

static int f8_matmul_common(const dmm::F8MatmulArgs& a, void* stream) {
    if (a.M < 0 || a.K < 0 || a.N < 0 || a.M >= kMaxDim || a.K >= dmm::kF8MaxK || a.N >= kMaxDim) return TQ_ERR_SHAPE;
    if (!is_dtype(a.y_dtype)) return TQ_ERR_DTYPE;
    if (a.M == 0 || a.N == 0) return TQ_OK;
    if (!a.y || (a.K > 0 && (!a.x_codes || !a.x_scales || !a.codes || !a.scales))) return TQ_ERR_NULL;
    if (!aligned(a.x_codes, 16) || !aligned(a.codes, 16) || !aligned(a.x_scales, 4) || !aligned(a.scales, 4) ||
        !aligned(a.bias, 4) || !aligned(a.y, bytes_of(a.y_dtype)))
        return TQ_ERR_ALIGN;
    return grid_status(dmm::launch_f8_matmul(a, (hipStream_t)stream));
}

int f8_matmul(const uint8_t* x_codes, const float* x_scales, int64_t M, int64_t K, const uint8_t* codes,
              const float* scales, int64_t N, const float* bias, void* y, int32_t y_dtype, void* stream) {
    const dmm::F8MatmulArgs a = {x_codes, x_scales, M,       K, N, codes,           scales,            bias,
                                 0,       nullptr,  nullptr, 1, y, plain(y_dtype), short_sums(y_dtype)};
    return f8_matmul_common(a, stream);
}

int f8_matmul_experts(const uint8_t* x_codes, const float* x_scales, int64_t M, int64_t K, const uint8_t* codes,
                      const float* scales, int64_t N, int32_t n_experts, const float* bias, const int32_t* offsets,
                      const int32_t* order, int32_t top_k, void* y, int32_t y_dtype, void* stream) {
    if (n_experts < 1 || top_k < 1) return TQ_ERR_SHAPE;
    if (M >= 0 && M < kMaxDim && M * top_k >= kMaxDim) return TQ_ERR_SHAPE;
    if (M > 0 && N > 0 && (!offsets || !order)) return TQ_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(order, 4)) return TQ_ERR_ALIGN;
    const dmm::F8MatmulArgs a = {x_codes,   x_scales, M,     K,     N, codes,           scales,            bias,
                                 n_experts, offsets,  order, top_k, y, plain(y_dtype), short_sums(y_dtype)};
    return f8_matmul_common(a, stream);
}

// ------------------------------------------- the experts' choice and combination

int moe_gate(const void* logits, int32_t l_dtype, int64_t M, int32_t n_experts, int64_t ldl,
             const uint8_t* token_mask, const float* bias, int32_t score, int32_t n_groups, int32_t top_groups,
             int32_t group_top, int32_t top_k, int32_t renorm, float scale, int32_t* expert_ids, float* weights,
             void* stream) {
    if (n_experts > dmm::kMoeMaxExperts || top_k > dmm::kGateMaxTopK || n_groups > 64) return TQ_ERR_UNSUPPORTED;
    if ((score != DMM_SOFTMAX && score != DMM_SIGMOID) || (group_top != 1 && group_top != 2)) return TQ_ERR_UNSUPPORTED;
    if (M < 0 || M >= kMaxDim || n_experts < 1 || !rows_ok(M, n_experts, ldl) || n_groups < 1 ||
        n_experts % n_groups != 0 || top_groups < 1 || top_groups > n_groups || top_k < 1 ||
        top_k > top_groups * (n_experts / n_groups))
        return TQ_ERR_SHAPE;
    if (!is_dtype(l_dtype)) return TQ_ERR_DTYPE;
    if (M == 0) return TQ_OK;
    if (!logits || !expert_ids || !weights) return TQ_ERR_NULL;
    if (!aligned(logits, bytes_of(l_dtype)) || !aligned(bias, 4) || !aligned(expert_ids, 4) || !aligned(weights, 4))
        return TQ_ERR_ALIGN;
    const dmm::GateArgs a = {logits,     l_dtype,   M,     n_experts,   ldl,   token_mask, bias,   score, n_groups,
                             top_groups, group_top, top_k, renorm != 0, scale, expert_ids, weights};
    return grid_status(dmm::launch_moe_gate(a, (hipStream_t)stream));
}

int moe_gate_grad(const void* logits, int32_t l_dtype, int64_t M, int32_t n_experts, int64_t ldl,
                  const int32_t* expert_ids, const float* dweights, int32_t score, int32_t top_k, int32_t renorm,
                  float scale, void* dlogits, void* stream) {
    if (n_experts > dmm::kMoeMaxExperts || top_k > dmm::kGateMaxTopK) return TQ_ERR_UNSUPPORTED;
    if (score != DMM_SOFTMAX && score != DMM_SIGMOID) return TQ_ERR_UNSUPPORTED;
    if (M < 0 || M >= kMaxDim || n_experts < 1 || !rows_ok(M, n_experts, ldl) || top_k < 1) return TQ_ERR_SHAPE;
    if (!is_dtype(l_dtype)) return TQ_ERR_DTYPE;
    if (M == 0) return TQ_OK;
    if (!logits || !expert_ids || !dweights || !dlogits) return TQ_ERR_NULL;
    if (!aligned(logits, bytes_of(l_dtype)) || !aligned(expert_ids, 4) || !aligned(dweights, 4) ||
        !aligned(dlogits, bytes_of(l_dtype)))
        return TQ_ERR_ALIGN;
    const dmm::GateGradArgs a = {logits, l_dtype, M,     n_experts,   ldl,   expert_ids, dweights,
                                 top_k,  score,   renorm != 0, scale, dlogits};
    return grid_status(dmm::launch_moe_gate_grad(a, (hipStream_t)stream));
}

int moe_combine(const void* y, int32_t y_dtype, int64_t M, int32_t top_k, int64_t N, const int32_t* expert_ids,
                const float* weights, int32_t n_experts, const void* add, void* out, int32_t out_dtype,
                void* stream) {
    if (M < 0 || N < 0 || M >= kMaxDim || N >= kMaxDim || top_k < 1 || M * top_k >= kMaxDim || n_experts < 1)
        return TQ_ERR_SHAPE;
    if (!is_dtype(y_dtype) || !is_dtype(out_dtype)) return TQ_ERR_DTYPE;
    if (M == 0 || N == 0) return TQ_OK;
    if (!y || !expert_ids || !weights || !out) return TQ_ERR_NULL;
    if (!aligned(y, bytes_of(y_dtype)) || !aligned(add, bytes_of(out_dtype)) || !aligned(out, bytes_of(out_dtype)) ||
        !aligned(expert_ids, 4) || !aligned(weights, 4))
        return TQ_ERR_ALIGN;
    const dmm::CombineArgs a = {y, y_dtype, M, top_k, N, expert_ids, weights, n_experts, add, out, out_dtype};
    return grid_status(dmm::launch_moe_combine(a, (hipStream_t)stream));
}

int moe_combine_grad(const void* y, int32_t y_dtype, int64_t M, int32_t top_k, int64_t N, const int32_t* expert_ids,
                     const float* weights, int32_t n_experts, const void* dout, int32_t dout_dtype, void* dy,
                     float* dweights, void* stream) {
    if (M < 0 || N < 0 || M >= kMaxDim || N >= kMaxDim || top_k < 1 || M * top_k >= kMaxDim || n_experts < 1)
        return TQ_ERR_SHAPE;
    if (!is_dtype(y_dtype) || !is_dtype(dout_dtype)) return TQ_ERR_DTYPE;
    if (M == 0) return TQ_OK;
    if (!expert_ids || !weights || !dweights || (N > 0 && (!y || !dout || !dy))) return TQ_ERR_NULL;
    if (!aligned(y, bytes_of(y_dtype)) || !aligned(dy, bytes_of(y_dtype)) || !aligned(dout, bytes_of(dout_dtype)) ||
        !aligned(expert_ids, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return TQ_ERR_ALIGN;
    const dmm::CombineGradArgs a = {y, y_dtype, M, top_k, N, expert_ids, weights, n_experts, dout, dout_dtype, dy, dweights};
    return grid_status(dmm::launch_moe_combine_grad(a, (hipStream_t)stream));
}

}  // extern "C"
