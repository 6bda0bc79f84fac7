// fp4q_internal.h -- argument bundles shared by the C-ABI layer and the
// kernel launchers of libfp4q.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp4q {

struct QuantArgs {
    const void *x;   // bf16 [rows x ld]
    int64_t rows, cols, ld;
    int axis;        // 0: along rows, 1: along columns (x^T)
    bool sr;
    bool hadamard;
    bool tiled;      // FP4Q_LAYOUT_TILED outputs
    uint64_t seed;
    uint32_t stream_id;
    uint32_t sign_mask;
    void *codes;
    void *scales;
    // dual output (axis 1 only): x along rows as well, rounded per rows_round
    // (0 none, 1 RNE, 2 SR) with its own stream id
    int rows_round;
    uint32_t stream_id_rows;
    void *codes_rows;
    void *scales_rows;
};

struct GemmArgs {
    const void *a_codes, *a_scales, *b_codes, *b_scales;
    const float *a_ts, *b_ts;  // NV tensor scales (null for MX)
    int nv_domain;             // NV only: 0 global, 1 tile128
    bool tiled;                // FP4Q_LAYOUT_TILED operands
    int64_t M, N, K;
    float alpha;
    void *c;
    bool c_bf16;
    int64_t ldc;
    uint32_t *c_amax;  // optional: max |C| as stored, folded in as binary32 bits
    // MX only, optional: C written as an MXFP4 operand along rows instead;
    // with q_swiglu, SwiGLU(C) (N / 2 columns: gate and up columns of C
    // interleaved in groups of 32)
    void *q_codes, *q_scales;
    bool q_tiled;
    bool q_swiglu;
};

struct DropoutArgs {
    const void *x, *residual;  // residual: optional
    int64_t rows, cols, ld_x, ld_r, ld_y;
    bool bf16;  // elements, else binary32
    float p;
    uint64_t seed;
    uint32_t stream_id;
    void *y;
};

struct NormArgs {
    const void *x, *residual;  // residual: optional
    int64_t rows, cols, ld_x, ld_r, ld_h, ld_y;
    int64_t rows_out;  // rows, or in the tiled MX layout rows rounded up to 32
    bool bf16;
    bool layer;  // else RMS
    const void *gamma, *beta;  // optional
    bool w_bf16;
    float eps, p;
    uint64_t seed;
    uint32_t stream_id;
    void *h, *y;         // optional
    float *mean, *rstd;  // optional
    void *codes, *scales;  // optional: the MXFP4 operand of a bf16 y
    bool tiled;
    void *codes8, *scales8;  // optional: y as 8-bit rows
};

struct NormGradArgs {
    const void *dy, *h, *dres;  // dres: optional
    const uint8_t *h_codes, *h_scales;  // h as 8-bit rows, in place of h
    int64_t rows, cols, ld_dy, ld_h, ld_dres, ld_dh, ld_dx;
    bool bf16;
    bool layer;
    const void *gamma;  // optional
    bool w_bf16;
    const float *mean, *rstd;
    float p;
    uint64_t seed;
    uint32_t stream_id;
    void *dh, *dx;  // one of them optional
    float *parts;   // workspace: the workgroups' weight sums
    uint32_t waves, groups, row_blocks;  // set by the launcher: waves of a row, rows of a workgroup, workgroups
};

struct SwigluGradArgs {
    const void *dh, *c;
    const uint8_t *c_codes, *c_scales;  // c as 8-bit rows, in place of c
    int64_t M, F, ld_dh, ldc, ld_dc, ldh, pair;
    void *dc, *h;  // h: optional
};

struct RotaryArgs {
    const void *x;
    int64_t tokens, x_token, x_head, y_token, y_head;
    uint32_t heads, dim, rot;
    bool bf16, interleaved, inverse, pos64;
    bool copy;  // the elements past rot have to be copied (y is not x)
    const void *positions;
    const float *inv_freq;
    float scale;
    void *y;
    uint32_t tokens_at_once;
};

struct Pack8Args {
    void *x;  // the rows, bf16 or binary32: read, or with `unpack` written
    int64_t rows, cols, ld;
    bool bf16, unpack;
    void *codes, *scales;
};

struct MatvecArgs {
    const void *x, *x_scales;  // bf16, or with x_scales the codes of 8-bit rows
    int64_t M, N, K, ld_x, ld_y;
    const void *codes, *scales;
    const float *tensor_scale;  // NV only
    int nv_domain;
    bool tiled;
    float alpha;
    void *y;
    bool y_bf16;
};

// Compute units of the current device (the persistent GEMMs' grid), looked
// up once per device; <= 0 if the device cannot be queried.
int device_cu_count();

int launch_quant_mx(const QuantArgs &a, hipStream_t st);
// given_amax: optional device pointer to the global domain's amax (skips the
// amax pass); null for the two-pass global path and the tile domain
int launch_quant_nv(const QuantArgs &a, int domain, float *tensor_scale, void *workspace, const float *given_amax,
                    hipStream_t st);
size_t nv_workspace_bytes(int domain);
int launch_gemm_mx(const GemmArgs &g, hipStream_t st);
int launch_gemm_nv(const GemmArgs &g, hipStream_t st);
// h[m][j] = bf16(SiLU(gate) * up) from a bf16 C whose columns interleave gate
// and up in groups of `pair` (a multiple of 8 dividing F)
int launch_swiglu(const void *c, int64_t M, int64_t F, int64_t ldc, int64_t pair, void *h, int64_t ldh,
                  hipStream_t st);
int launch_dropout(const DropoutArgs &a, hipStream_t st);
int launch_norm(const NormArgs &a, hipStream_t st);
size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols, bool bf16);
int launch_norm_grad(const NormGradArgs &a, float *dgamma, float *dbeta, hipStream_t st);
// its rows' part where h comes as 8-bit rows
int norm_grad_rows_pack8(const NormGradArgs &a, float *dgamma, float *dbeta, hipStream_t st);
int launch_swiglu_grad(const SwigluGradArgs &a, hipStream_t st);
int launch_rotary(RotaryArgs a, hipStream_t st);
int launch_pack8(const Pack8Args &a, hipStream_t st);
int launch_matvec_zero(const MatvecArgs &a, hipStream_t st);  // K == 0: only M, N and Y are looked at
int launch_matvec_mx(const MatvecArgs &a, hipStream_t st);
int launch_matvec_nv(const MatvecArgs &a, hipStream_t st);

}  // namespace fp4q
