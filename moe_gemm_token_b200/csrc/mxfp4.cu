// MXFP4 (OCP Microscaling specification 1.0) on sm_100a: E2M1 codes with one
// power-of-two scale (E8M0) per 32 elements. Quantization, reading back, and
// the product of two MXFP4 matrices.
#include "common.cuh"
#include "../../include/metis_mxfp4.h"

namespace metis {
namespace mxfp4 {

// Byte offset of the scale of row r, block b in the tiled layout (kc = K / 128 atoms per 128 rows).
__host__ __device__ __forceinline__ int64_t tiled_offset(int64_t r, int64_t b, int64_t kc) {
    return ((r >> 7) * kc + (b >> 2)) * 512 + 16 * (r & 31) + 4 * ((r & 127) >> 5) + (b & 3);
}

__device__ __forceinline__ float load_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_value(const float* p) { return *p; }

__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, b, b, b};\n\t}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r & 0xFFu;
}

__device__ __forceinline__ float e2m1_value(uint32_t n) {
    const float mag = (n & 6u) == 0 ? 0.5f * (n & 1u) : (1.0f + 0.5f * (n & 1u)) * static_cast<float>(1u << ((n >> 1 & 3u) - 1u));
    return n & 8u ? -mag : mag;
}

__device__ __forceinline__ float e8m0_value(uint32_t c) {
    if (c == 255u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(c == 0 ? 0x00400000u : c << 23);
}

// Scale code of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;  // an infinity or a NaN in the block
    const int e = static_cast<int>(amax_bits >> 23) - 2;  // a subnormal amax is below 2^-126: clamped to code 0
    return e < 0 ? 0u : static_cast<uint32_t>(e);
}

// One thread per block of 32 elements.
template <typename T>
__global__ void __launch_bounds__(256) quant_kernel(const T* x, int64_t R, int64_t K, int64_t ldx, uint8_t* q,
                                                    uint8_t* sf, int tiled, int64_t rows) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t nb = K / 32;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= rows * nb) return;
    const int64_t r = i / nb, b = i - r * nb;
    const int64_t at = tiled ? tiled_offset(r, b, K / 128) : i;
    if (r >= R) {
        sf[at] = 0;
        return;
    }
    const T* p = x + r * ldx + 32 * b;
    uint32_t m = 0;
    for (int k = 0; k < 32; ++k) m = max(m, __float_as_uint(load_value(p + k)) & 0x7FFFFFFFu);
    const uint32_t c = scale_code(m);
    const float inv = c == 255u ? 0.0f : __uint_as_float((254u - c) << 23);
    for (int k = 0; k < 32; k += 2) {
        const float v0 = __fmul_rn(load_value(p + k), inv), v1 = __fmul_rn(load_value(p + k + 1), inv);
        q[(r * K + 32 * b + k) / 2] = static_cast<uint8_t>(c == 255u ? 0u : e2m1_pair(v0, v1));
    }
    sf[at] = static_cast<uint8_t>(c);
}

__global__ void __launch_bounds__(256) dequant_kernel(const uint8_t* q, const uint8_t* sf, int tiled, int64_t R,
                                                      int64_t K, __nv_bfloat16* y) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t nb = K / 32;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= R * nb) return;
    const int64_t r = i / nb, b = i - r * nb;
    const float s = e8m0_value(sf[tiled ? tiled_offset(r, b, K / 128) : i]);
    for (int k = 0; k < 32; ++k) {
        const uint8_t byte = q[(r * K + 32 * b + k) / 2];
        y[r * K + 32 * b + k] = __float2bfloat16_rn(__fmul_rn(e2m1_value(k & 1 ? byte >> 4 : byte & 15u), s));
    }
}

// One warp per output.
__global__ void __launch_bounds__(256) gemm_kernel(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb,
                                                   const uint8_t* sfb, int N, int K, int64_t m0, __nv_bfloat16* y) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int n = blockIdx.x * 8 + threadIdx.x / 32;
    const int64_t m = m0 + blockIdx.y;
    if (n >= N) return;
    float acc = 0.0f;
    for (int j = lane; j < K / 2; j += 32) {
        const uint32_t a = qa[m * (K / 2) + j], b = qb[static_cast<int64_t>(n) * (K / 2) + j];
        const float s = e8m0_value(sfa[tiled_offset(m, j / 16, K / 128)]) * e8m0_value(sfb[tiled_offset(n, j / 16, K / 128)]);
        acc = fmaf(e2m1_value(a & 15u) * e2m1_value(b & 15u) + e2m1_value(a >> 4) * e2m1_value(b >> 4), s, acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) y[m * N + n] = __float2bfloat16_rn(acc);
}

int check_rows(const char* name, int64_t R, int64_t K, int layout) {
    if (layout != METIS_SF_ROWMAJOR && layout != METIS_SF_TILED)
        return fail(METIS_ERR_INVALID_ARG, "%s: sf_layout %d", name, layout);
    if (R < 0 || R > 0x7fffffffll || K < 32 || K % 32 || K > 65536 || (layout == METIS_SF_TILED && K % 128))
        return fail(METIS_ERR_INVALID_ARG,
                    "%s: need R >= 0, 32 <= K <= 65536 with K %% 32 == 0 (tiled scales: K %% 128 == 0) "
                    "(R=%lld K=%lld)", name, (long long)R, (long long)K);
    return METIS_OK;
}

}  // namespace mxfp4
}  // namespace metis

using namespace metis;

extern "C" int metis_quant_mxfp4(const void* x, int x_kind, int64_t R, int64_t K, int64_t ldx, uint8_t* q,
                                 uint8_t* sf, int sf_layout, metis_stream_t stream) {
    using namespace mxfp4;
    clear_error();
    if (x_kind != METIS_A_BF16 && x_kind != METIS_A_F32)
        return fail(METIS_ERR_INVALID_ARG, "quant_mxfp4: x_kind %d (need METIS_A_BF16 or METIS_A_F32)", x_kind);
    int rc = check_rows("quant_mxfp4", R, K, sf_layout);
    if (rc) return rc;
    if (ldx < K) return fail(METIS_ERR_INVALID_ARG, "quant_mxfp4: ldx=%lld below K=%lld", (long long)ldx, (long long)K);
    if (R == 0) return METIS_OK;
    if (!x || !q || !sf) return fail(METIS_ERR_INVALID_ARG, "quant_mxfp4: null pointer");
    const int tiled = sf_layout == METIS_SF_TILED;
    if (!aligned(x, 16) || (ldx * (x_kind == METIS_A_BF16 ? 2 : 4)) % 16 || !aligned(q, 16) ||
        (tiled && !aligned(sf, 4)))
        return fail(METIS_ERR_INVALID_ARG,
                    "quant_mxfp4: x and q 16-byte aligned, ldx * element size a multiple of 16, tiled sf 4-byte aligned");
    DeviceInfo di;
    if ((rc = current_device_info(&di))) return rc;
    const int64_t rows = tiled ? (R + 127) / 128 * 128 : R;
    const unsigned grid = static_cast<unsigned>((rows * (K / 32) + 255) / 256);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_kind == METIS_A_BF16)
        return cuda_check(launch_pdl(quant_kernel<__nv_bfloat16>, dim3(grid), dim3(256), 0, st, 1,
                                     static_cast<const __nv_bfloat16*>(x), R, K, ldx, q, sf, tiled, rows),
                          "quant_mxfp4 launch");
    return cuda_check(launch_pdl(quant_kernel<float>, dim3(grid), dim3(256), 0, st, 1, static_cast<const float*>(x), R,
                                 K, ldx, q, sf, tiled, rows),
                      "quant_mxfp4 launch");
}

extern "C" int metis_dequant_mxfp4(const uint8_t* q, const uint8_t* sf, int sf_layout, int64_t R, int64_t K,
                                   void* y_bf16, metis_stream_t stream) {
    using namespace mxfp4;
    clear_error();
    int rc = check_rows("dequant_mxfp4", R, K, sf_layout);
    if (rc || R == 0) return rc;
    if (!q || !sf || !y_bf16) return fail(METIS_ERR_INVALID_ARG, "dequant_mxfp4: null pointer");
    const int tiled = sf_layout == METIS_SF_TILED;
    if (!aligned(q, 16) || !aligned(y_bf16, 16) || (tiled && !aligned(sf, 4)))
        return fail(METIS_ERR_INVALID_ARG, "dequant_mxfp4: q and y 16-byte aligned, tiled sf 4-byte aligned");
    DeviceInfo di;
    if ((rc = current_device_info(&di))) return rc;
    const unsigned grid = static_cast<unsigned>((R * (K / 32) + 255) / 256);
    return cuda_check(launch_pdl(dequant_kernel, dim3(grid), dim3(256), 0, static_cast<cudaStream_t>(stream), 1, q, sf,
                                 tiled, R, K, static_cast<__nv_bfloat16*>(y_bf16)),
                      "dequant_mxfp4 launch");
}

extern "C" int metis_mxfp4_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb,
                                void* y_bf16, int64_t M, int64_t N, int64_t K, metis_stream_t stream) {
    using namespace mxfp4;
    clear_error();
    if (M < 0 || M > (1ll << 30) || N < 128 || N % 128 || N > (1 << 20) || K < 128 || K % 128 || K > 65536)
        return fail(METIS_ERR_INVALID_ARG,
                    "mxfp4_gemm: need M >= 0, N and K multiples of 128, K in [128, 65536] "
                    "(M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
    if (M == 0) return METIS_OK;
    if (!qa || !sfa || !qb || !sfb || !y_bf16) return fail(METIS_ERR_INVALID_ARG, "mxfp4_gemm: null pointer");
    if (!aligned(qa, 16) || !aligned(sfa, 16) || !aligned(qb, 16) || !aligned(sfb, 16) || !aligned(y_bf16, 16))
        return fail(METIS_ERR_INVALID_ARG, "mxfp4_gemm: codes, tiled scales and y 16-byte aligned");
    DeviceInfo di;
    int rc = current_device_info(&di);
    if (rc) return rc;
    for (int64_t m = 0; m < M; m += 65535) {
        const unsigned rows = static_cast<unsigned>(M - m < 65535 ? M - m : 65535);
        rc = cuda_check(launch_pdl(gemm_kernel, dim3(static_cast<unsigned>((N + 7) / 8), rows), dim3(256), 0,
                                   static_cast<cudaStream_t>(stream), 1, qa, sfa, qb, sfb, static_cast<int>(N),
                                   static_cast<int>(K), m, static_cast<__nv_bfloat16*>(y_bf16)),
                        "mxfp4_gemm launch");
        if (rc) return rc;
    }
    return METIS_OK;
}
