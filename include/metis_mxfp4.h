/*
 * metis_mxfp4.h — C ABI of the MXFP4 operators of libmetis_fp8 (B200, sm_100a):
 * quantization to the 4-bit microscaling format of the OCP Microscaling (MX)
 * specification 1.0, reading values back, and the product of two MXFP4
 * matrices on the FP4 tensor cores. They stand beside the NVFP4 operators of
 * metis_nvfp4.h, whose codes they share; the scales differ.
 *
 * Definitions:
 *  - E2M1 codes: as in metis_nvfp4.h, two per byte, element 2i in the low nibble.
 *  - block scale: one E8M0 byte c per 32 consecutive elements of a row, worth
 *    2^(c - 127); 255 is NaN.
 *  - quantization of a block with largest magnitude amax:
 *      c = clamp(floor(log2(amax)) - 2, -127, 125) + 127, 0 for an all-zero block;
 *      code = E2M1_rn_satfinite(x * 2^(127 - c)), ties to the even code (a
 *      value between 6 and 8 steps saturates to 6); a zero keeps its sign.
 *    A block that holds an infinity or a NaN gets c = 255 and zero codes, so
 *    that every value of the block reads back as NaN.
 *  - product: y[m, n] = bf16_rn( sum_k V_a[m, k] V_b[n, k] ), V = D2(code) * 2^(c - 127),
 *    FP32 accumulation.
 *  - scale layouts: METIS_SF_ROWMAJOR [R, K/32], and METIS_SF_TILED, the
 *    tensor cores' order [ceil(R/128)][K/128][512]: the 512-byte atom of rows
 *    128 a .. 128 a + 127 and elements 128 c .. 128 c + 127 holds the scale of
 *    row 128 a + r, block 4 c + j at byte 16 (r % 32) + 4 (r / 32) + j.
 *
 * Conventions are those of metis_fp8.h: device pointers owned by the caller,
 * nothing allocated or synchronised, asynchronous on `stream`, METIS_OK or a
 * negative metis_status with argument errors found before any launch,
 * bounded device waits, bitwise reproducible results. Outputs overlap no
 * other argument.
 */
#ifndef METIS_MXFP4_H
#define METIS_MXFP4_H

#include "metis_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * MXFP4 quantization of R rows of K elements.
 *   x   [R, ldx] BF16 bit patterns (x_kind METIS_A_BF16) or FP32 (METIS_A_F32);
 *       16-byte aligned, ldx * element size a multiple of 16.
 *   q   [R, K/2] packed codes (16-byte aligned).
 *   sf  block scales in `sf_layout`; METIS_SF_TILED needs K % 128 == 0 and
 *       ceil(R/128) * 128 * K/32 bytes, 4-byte aligned (the pad rows of the
 *       last 128 are written as 0, which is 2^-127).
 * K: a multiple of 32, 32 <= K <= 65536. R >= 0 (0: nothing launched).
 */
METIS_API int metis_quant_mxfp4(const void* x, int x_kind, int64_t R, int64_t K, int64_t ldx, uint8_t* q,
                                uint8_t* sf, int sf_layout, metis_stream_t stream);

/*
 * y [R, K] = the values of MXFP4 codes q [R, K/2] and block scales sf (row-
 * major [R, K/32] or tiled), as BF16. Exact for scale codes up to 252, which
 * is all that metis_quant_mxfp4 writes; a value past BF16's range becomes an
 * infinity, a scale code of 255 NaN. K and R as above; q and y 16-byte
 * aligned, tiled scales 4-byte aligned.
 */
METIS_API int metis_dequant_mxfp4(const uint8_t* q, const uint8_t* sf, int sf_layout, int64_t R, int64_t K,
                                  void* y_bf16, metis_stream_t stream);

/*
 * y [M, N] = MXFP4 product (above) on the tensor cores.
 *   qa  [ceil(M/128) * 128, K/2] packed codes of A: the rows past M are read
 *       (their results are discarded), so the buffer must hold them.
 *   sfa tiled block scales of A (ceil(M/128) atoms of rows).
 *   qb  [N, K/2] packed codes of B (output channel n = row n); sfb its tiled scales.
 *   y   [M, N] BF16, row-major.
 * K and N multiples of 128, 128 <= K <= 65536, N <= 2^20; 0 <= M <= 2^30.
 * Codes, tiled scales and y 16-byte aligned.
 */
METIS_API int metis_mxfp4_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb,
                               void* y_bf16, int64_t M, int64_t N, int64_t K, metis_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* METIS_MXFP4_H */
