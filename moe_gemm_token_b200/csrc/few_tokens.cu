// Default maths for few tokens with the weights read once: the routed-expert
// layer with FP8 or NVFP4 experts, and the NVFP4 weight-only product.
//   h[s] = W_up[e] x[t],  o[s] = W_down[e] h[s],  y[t] = bf16( sum_j w[t, j] o[t, j] )
// for the slots s = (t, j) with expert e = topk_ids[t, j]; FP32 sums, h and o
// kept in FP32.
#include "common.cuh"
#include "../../include/metis_nvfp4.h"

namespace metis {
namespace few {

constexpr int MAX_T = 128;       // tokens of a routed layer
constexpr int MAX_S = 1024;      // slots (T * topk)
constexpr int MAX_E = 1024;
constexpr int MAX_K = 8192;      // H and I of a routed layer

enum Fmt { FP8 = 0, NVFP4 = 1 };

// One expert matrix set: E matrices of N rows by K.
struct Weights {
    const uint8_t* q;     // FP8: [E * N, K] codes; NVFP4: [E * N, K / 2]
    const uint8_t* sf;    // NVFP4: tiled block scales of the [E * N, K] matrix
    const float* s;       // FP8: [E * N] channel scales; NVFP4: [E] global scales
    int N, K;
};

__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h;
    asm("{\n\t.reg .b16 q;\n\tcvt.u16.u32 q, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, q;\n\t}" : "=r"(h) : "r"(code & 0xFFu));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

__device__ __forceinline__ float e2m1_value(uint32_t n) {
    const float mag = (n & 6u) == 0 ? 0.5f * (n & 1u) : (1.0f + 0.5f * (n & 1u)) * static_cast<float>(1u << ((n >> 1 & 3u) - 1u));
    return n & 8u ? -mag : mag;
}

template <int FMT>
__device__ __forceinline__ float weight(const Weights& w, int64_t row, int k) {
    if constexpr (FMT == FP8) return e4m3_value(w.q[row * w.K + k]);
    const uint8_t b = w.q[row * (w.K / 2) + k / 2];
    const int64_t atom = (row >> 7) * (w.K / 64) + k / 64;
    const uint8_t s = w.sf[atom * 512 + 16 * (row & 31) + 4 * ((row & 127) >> 5) + (k % 64) / 16];
    return e2m1_value(k & 1 ? b >> 4 : b & 15u) * e4m3_value(s);
}

__device__ __forceinline__ float in_value(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float in_value(const float* p, int64_t i) { return p[i]; }

// One warp per (slot, weight row): out[slot][n] = scale * sum_k in[row(slot)][k] w[e][n][k].
template <int FMT, typename In, typename Out>
__global__ void __launch_bounds__(256) rows_kernel(const In* in, int in_div, const Weights w, const int32_t* ids,
                                                   int E, Out* out, uint32_t* status) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int n = blockIdx.x * 8 + threadIdx.x / 32;
    const int slot = blockIdx.y;
    const int e = ids ? ids[slot] : 0;
    if (e < 0 || e >= E) {
        if (lane == 0 && n == 0) atomicOr(status, kDevErrBadIndex);
        return;
    }
    if (n >= w.N) return;
    const int64_t row = static_cast<int64_t>(e) * w.N + n;
    const In* x = in + static_cast<int64_t>(slot / in_div) * w.K;
    float acc = 0.0f;
    for (int k = lane; k < w.K; k += 32) acc = fmaf(in_value(x, k), weight<FMT>(w, row, k), acc);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) {
        const float v = acc * w.s[FMT == FP8 ? row : e];
        if constexpr (sizeof(Out) == 2) out[static_cast<int64_t>(slot) * w.N + n] = __float2bfloat16_rn(v);
        else out[static_cast<int64_t>(slot) * w.N + n] = v;
    }
}

// y[t] = bf16( sum_j w[t, j] o[t, j] ), FP32, j ascending; slots of no expert add nothing.
__global__ void __launch_bounds__(256) combine_kernel(const float* o, const int32_t* ids, const float* tw, int topk,
                                                      int E, int H, __nv_bfloat16* y) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int n = blockIdx.x * 256 + threadIdx.x;
    const int t = blockIdx.y;
    if (n >= H) return;
    float acc = 0.0f;
    for (int j = 0; j < topk; ++j) {
        const int s = t * topk + j;
        if (ids[s] >= 0 && ids[s] < E) acc = fmaf(tw[s], o[static_cast<int64_t>(s) * H + n], acc);
    }
    y[static_cast<int64_t>(t) * H + n] = __float2bfloat16_rn(acc);
}

inline int64_t align256(int64_t v) { return (v + 255) & ~static_cast<int64_t>(255); }

// The argument checks that the two routed layers share (`step`: what H and I
// are multiples of).
int check_moe(const char* name, int act, int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I, int step) {
    if (act != METIS_ACT_NONE)
        return fail(METIS_ERR_UNSUPPORTED, "%s: act %d (only METIS_ACT_NONE)", name, act);
    if (T < 0 || topk < 1 || E < 1 || E > MAX_E || topk > E || H < step || H % step || H > MAX_K || I < step ||
        I % step || I > MAX_K)
        return fail(METIS_ERR_INVALID_ARG,
                    "%s: need T >= 0, 1 <= topk <= E <= %d, H and I multiples of %d in [%d, %d] "
                    "(T=%lld topk=%lld E=%lld H=%lld I=%lld)", name, MAX_E, step, step, MAX_K, (long long)T,
                    (long long)topk, (long long)E, (long long)H, (long long)I);
    if (T > MAX_T || T * topk > MAX_S)
        return fail(METIS_ERR_UNSUPPORTED,
                    "%s: made for few tokens, T <= %d and T * topk <= %d (T=%lld topk=%lld); use the grouped "
                    "GEMM layer for more", name, MAX_T, MAX_S, (long long)T, (long long)topk);
    return METIS_OK;
}

template <int FMT>
int run_moe(const __nv_bfloat16* x, const int32_t* ids, const float* tw, int T, int topk, int E, const Weights& up,
            const Weights& down, __nv_bfloat16* y, uint8_t* ws, cudaStream_t st) {
    uint32_t* status = nullptr;
    int rc = device_status_word(&status);
    if (rc) return rc;
    const int S = T * topk;
    float* h = reinterpret_cast<float*>(ws);
    float* o = reinterpret_cast<float*>(ws + align256(4ll * S * up.N));
    if ((rc = cuda_check(launch_pdl(rows_kernel<FMT, __nv_bfloat16, float>, dim3((up.N + 7) / 8, S), dim3(256), 0, st,
                                    1, x, topk, up, ids, E, h, status),
                         "few-token up-projection launch")))
        return rc;
    if ((rc = cuda_check(launch_pdl(rows_kernel<FMT, float, float>, dim3((down.N + 7) / 8, S), dim3(256), 0, st, 1,
                                    static_cast<const float*>(h), 1, down, ids, E, o, status),
                         "few-token down-projection launch")))
        return rc;
    return cuda_check(launch_pdl(combine_kernel, dim3((down.N + 255) / 256, T), dim3(256), 0, st, 1,
                                 static_cast<const float*>(o), ids, tw, topk, E, down.N, y),
                      "few-token combine launch");
}

}  // namespace few

// Bytes of the routed layers' workspace: h [S, I] and o [S, H], FP32.
size_t few_moe_workspace(int64_t T, int64_t topk, int64_t H, int64_t I) {
    return static_cast<size_t>(few::align256(4 * T * topk * I) + few::align256(4 * T * topk * H));
}

}  // namespace metis

using namespace metis;

extern "C" int metis_moe_w8a16(const void* x_bf16, const int32_t* topk_ids, const float* topk_w, int64_t T,
                               int64_t topk, int64_t E, int64_t H, int64_t I, const uint8_t* w_up,
                               const float* s_up, const uint8_t* w_down, const float* s_down, int act, void* y_bf16,
                               void* workspace, size_t ws_bytes, metis_stream_t stream) {
    clear_error();
    int rc = few::check_moe("moe_w8a16", act, T, topk, E, H, I, 16);
    if (rc || T == 0) return rc;
    if (!x_bf16 || !topk_ids || !topk_w || !w_up || !s_up || !w_down || !s_down || !y_bf16)
        return fail(METIS_ERR_INVALID_ARG, "moe_w8a16: null pointer");
    if (!aligned(x_bf16, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || !aligned(y_bf16, 16) ||
        !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(s_up, 4) || !aligned(s_down, 4))
        return fail(METIS_ERR_INVALID_ARG, "moe_w8a16: x, weights and y must be 16-byte aligned");
    const size_t need = metis_workspace_size(METIS_OP_MOE_W8A16, T, I, H, topk, E);
    if (!workspace || ws_bytes < need || !aligned(workspace, 256))
        return fail(METIS_ERR_INVALID_ARG, "moe_w8a16: needs a 256-byte aligned workspace of %zu bytes (got %zu)",
                    need, ws_bytes);
    DeviceInfo di;
    if ((rc = current_device_info(&di))) return rc;
    const few::Weights up{w_up, nullptr, s_up, static_cast<int>(I), static_cast<int>(H)};
    const few::Weights down{w_down, nullptr, s_down, static_cast<int>(H), static_cast<int>(I)};
    return few::run_moe<few::FP8>(static_cast<const __nv_bfloat16*>(x_bf16), topk_ids, topk_w, static_cast<int>(T),
                                  static_cast<int>(topk), static_cast<int>(E), up, down,
                                  static_cast<__nv_bfloat16*>(y_bf16), static_cast<uint8_t*>(workspace),
                                  static_cast<cudaStream_t>(stream));
}

extern "C" int metis_moe_nvfp4_w4a16(const void* x_bf16, const int32_t* topk_ids, const float* topk_w, int64_t T,
                                     int64_t topk, int64_t E, int64_t H, int64_t I, const uint8_t* w_up,
                                     const uint8_t* sf_up, const float* g_up, const uint8_t* w_down,
                                     const uint8_t* sf_down, const float* g_down, int act, void* y_bf16,
                                     void* workspace, size_t ws_bytes, metis_stream_t stream) {
    clear_error();
    int rc = few::check_moe("moe_nvfp4_w4a16", act, T, topk, E, H, I, 128);
    if (rc || T == 0) return rc;
    if (!x_bf16 || !topk_ids || !topk_w || !w_up || !sf_up || !g_up || !w_down || !sf_down || !g_down || !y_bf16)
        return fail(METIS_ERR_INVALID_ARG, "moe_nvfp4_w4a16: null pointer");
    if (!aligned(x_bf16, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || !aligned(y_bf16, 16) ||
        !aligned(sf_up, 16) || !aligned(sf_down, 16) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
        !aligned(g_up, 4) || !aligned(g_down, 4))
        return fail(METIS_ERR_INVALID_ARG, "moe_nvfp4_w4a16: x, weights, tiled scales and y must be 16-byte aligned");
    const size_t need = metis_workspace_size(METIS_OP_MOE_NVFP4_W4A16, T, I, H, topk, E);
    if (!workspace || ws_bytes < need || !aligned(workspace, 256))
        return fail(METIS_ERR_INVALID_ARG,
                    "moe_nvfp4_w4a16: needs a 256-byte aligned workspace of %zu bytes (got %zu)", need, ws_bytes);
    DeviceInfo di;
    if ((rc = current_device_info(&di))) return rc;
    const few::Weights up{w_up, sf_up, g_up, static_cast<int>(I), static_cast<int>(H)};
    const few::Weights down{w_down, sf_down, g_down, static_cast<int>(H), static_cast<int>(I)};
    return few::run_moe<few::NVFP4>(static_cast<const __nv_bfloat16*>(x_bf16), topk_ids, topk_w, static_cast<int>(T),
                                    static_cast<int>(topk), static_cast<int>(E), up, down,
                                    static_cast<__nv_bfloat16*>(y_bf16), static_cast<uint8_t*>(workspace),
                                    static_cast<cudaStream_t>(stream));
}

extern "C" int metis_nvfp4_w4a16_gemm(const void* x_bf16, const uint8_t* qb, const uint8_t* sfb, const float* gb,
                                      void* y_bf16, int64_t M, int64_t N, int64_t K, void* workspace,
                                      size_t ws_bytes, metis_stream_t stream) {
    clear_error();
    if (M < 0 || M > 0x7fffffff || N < 128 || N % 128 || N > (1 << 20) || K < 64 || K % 64 || K > 65536)
        return fail(METIS_ERR_INVALID_ARG,
                    "nvfp4_w4a16_gemm: need M >= 0, N a multiple of 128, K a multiple of 64 in [64, 65536] "
                    "(M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
    if (M == 0) return METIS_OK;
    if (!x_bf16 || !qb || !sfb || !gb || !y_bf16)
        return fail(METIS_ERR_INVALID_ARG, "nvfp4_w4a16_gemm: null pointer");
    if (!aligned(x_bf16, 16) || !aligned(qb, 16) || !aligned(sfb, 16) || !aligned(y_bf16, 16) || !aligned(gb, 4))
        return fail(METIS_ERR_INVALID_ARG, "nvfp4_w4a16_gemm: x, codes, tiled scales and y 16-byte aligned");
    const size_t need = metis_workspace_size(METIS_OP_NVFP4_W4A16, M, N, K, 0, 0);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return fail(METIS_ERR_INVALID_ARG,
                    "nvfp4_w4a16_gemm: needs a 256-byte aligned workspace of %zu bytes (got %zu)", need, ws_bytes);
    DeviceInfo di;
    int rc = current_device_info(&di);
    if (rc) return rc;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status))) return rc;
    const few::Weights w{qb, sfb, gb, static_cast<int>(N), static_cast<int>(K)};
    // grid.y holds at most 65,535 rows
    for (int64_t m = 0; m < M; m += 65535) {
        const unsigned rows = static_cast<unsigned>(M - m < 65535 ? M - m : 65535);
        rc = cuda_check(launch_pdl(few::rows_kernel<few::NVFP4, __nv_bfloat16, __nv_bfloat16>,
                                   dim3(static_cast<unsigned>((N + 7) / 8), rows), dim3(256), 0,
                                   static_cast<cudaStream_t>(stream), 1,
                                   static_cast<const __nv_bfloat16*>(x_bf16) + m * K, 1, w,
                                   static_cast<const int32_t*>(nullptr), 1, static_cast<__nv_bfloat16*>(y_bf16) + m * N,
                                   status),
                        "nvfp4_w4a16_gemm launch");
        if (rc) return rc;
    }
    return METIS_OK;
}
