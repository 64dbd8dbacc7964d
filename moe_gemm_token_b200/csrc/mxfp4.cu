// MXFP4 (OCP Microscaling specification 1.0) on sm_100a: E2M1 codes with one
// power-of-two scale (E8M0) per 32 elements. Quantization and reading back
// here; the product of two MXFP4 matrices is the block-scaled GEMM of
// nvfp4.cu with kind::mxf4.
#include "common.cuh"
#include "../../include/metis_mxfp4.h"

namespace metis {
namespace mxfp4 {

// Byte offset of the scale of row r, block b in the tiled layout (kc = K / 128 atoms per 128 rows).
__host__ __device__ __forceinline__ int64_t tiled_offset(int64_t r, int64_t b, int64_t kc) {
    return ((r >> 7) * kc + (b >> 2)) * 512 + 16 * (r & 31) + 4 * ((r & 127) >> 5) + (b & 3);
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

// 32 bytes (a whole sector) by one load or store at a 32-byte aligned address.
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.u32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// Half a block, 16 consecutive elements: a lane's share. Two lanes make a
// block, eight a group of four blocks (128 elements, whose scales are one
// 32-bit word in both layouts).
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16* p, bool wide) {
        if (wide) {
            load32(p, w);
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
    }
    // bits of the largest magnitude, as binary32 (an infinity or a NaN is above all others)
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return max(m & 0xFFFF0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <>
struct Half<float> {
    uint32_t w[2][8];
    __device__ __forceinline__ void load(const float* p, bool wide) {
        if (wide) {
            load32(p, w[0]);
            load32(p + 8, w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
                uint32_t* o = &w[i / 2][4 * (i % 2)];
                o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
            }
        }
    }
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, w[i / 8][i % 8] & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i / 8][i % 8]);
    }
};

// Two binary32 values -> their E2M1 codes (nearest even, saturating; lo in
// bits 0..3) in every byte.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, b, b, b};\n\t}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// Eight values -> eight codes, v[0] in bits 0..3. The four bytes are joined
// with byte permutations: one mov of four different .b8 registers came out
// with three of them zero here (CUDA 12.9).
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
    const uint32_t lo = __byte_perm(e2m1x2(v[0], v[1]), e2m1x2(v[2], v[3]), 0x4040);
    const uint32_t hi = __byte_perm(e2m1x2(v[4], v[5]), e2m1x2(v[6], v[7]), 0x4040);
    return __byte_perm(lo, hi, 0x5410);
}
// Eight E2M1 codes times an FP32 scale -> eight BF16 values.
__device__ __forceinline__ uint4 e2m1x8_to_bf16(uint32_t w, float s) {
    uint32_t h[4], o[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        o[i] = pack_bf16x2(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int THREADS = 256;
// Halves of a lane in flight, and blocks per SM: all resident at once, each
// thread looping over its share. Quantizing 8192 x 8192 BF16 (us): 2 halves
// 33.7, 3 halves 33.0, 4 halves 36.3, 8 halves (2 blocks) 38.1; 5 or 6 blocks
// 33.9 to 37.5. 8192 x 4096 FP32: 2 halves 26.0.
template <typename T>
constexpr int batch() { return sizeof(T) == 2 ? 3 : 2; }
constexpr int BATCH = 4, PER_SM = 4, DEQUANT_PER_SM = 8;

// n / d for d > 0 with inv = floor((2^32 - 1) / d), n < 2^32: at most one short.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t d, uint32_t inv, uint32_t& rest) {
    uint32_t q = __umulhi(n, inv);
    rest = n - q * d;
    if (rest >= d) ++q, rest -= d;
    return q;
}

struct RowArgs {
    const void* x;       // quant: rows of ldx elements; dequant: null
    uint8_t* q;          // [R, K / 2]
    uint8_t* sf;
    __nv_bfloat16* y;    // dequant: [R, K]
    int64_t ldx;
    uint32_t R, halves, inv;  // rows, halves per row (K / 16), for divide()
    int64_t total;            // halves of all rows (quant, tiled: with the pad rows)
    int tiled, groups;        // tiled scales; K a multiple of 128
    int wide;                 // every half (quant: of x, dequant: of y) starts on 32 bytes
};

// Scale byte offset of half h of row r.
__device__ __forceinline__ int64_t scale_offset(const RowArgs& a, uint32_t r, uint32_t h) {
    return a.tiled ? tiled_offset(r, h >> 1, a.halves >> 3) : static_cast<int64_t>(r) * (a.halves >> 1) + (h >> 1);
}

// A lane quantizes one half at a time. HBM-bound: 2 bytes read and 17/32
// written per BF16 element; a warp reads 1 KB and writes 256 + 16 bytes of
// consecutive memory per step, BATCH steps in flight. 8192 x 8192 BF16: 33.0
// us, 5.1 TB/s; 8192 x 4096 FP32: 26.0 us, 5.8 TB/s.
template <typename T>
__global__ void __launch_bounds__(THREADS, PER_SM) quant_kernel(const RowArgs a) {
    constexpr int BATCH = batch<T>();
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * THREADS;
    const int lane = threadIdx.x % 32;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i0 - lane < a.total; i0 += BATCH * stride) {
        Half<T> x[BATCH];
        uint32_t r[BATCH], h[BATCH];
        bool live[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t i = i0 + b * stride;
            const bool in = i < a.total;
            r[b] = divide(static_cast<uint32_t>(in ? i : 0), a.halves, a.inv, h[b]);
            live[b] = in && r[b] < a.R;
            if (live[b]) x[b].load(static_cast<const T*>(a.x) + r[b] * a.ldx + 16 * h[b], a.wide);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            uint32_t m = live[b] ? x[b].amax() : 0u;
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));  // the block's other half
            uint32_t c = live[b] ? scale_code(m) : 0u;       // the pad rows' scales are 0
            if (live[b]) {
                const float inv = __uint_as_float((254u - c) << 23);  // 2^(127 - c)
                float v[16];
                x[b].get(v);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __fmul_rn(v[k], inv);
                uint2 o = make_uint2(e2m1x8(v), e2m1x8(v + 8));
                if (c == 255u) o = make_uint2(0, 0);
                *reinterpret_cast<uint2*>(a.q + (static_cast<int64_t>(r[b]) * a.halves + h[b]) * 8) = o;
            }
            const bool in = i0 + b * stride < a.total;
            if (a.groups) {
                // four blocks' scales in one word: lanes 0, 2, 4, 6 of each eight
                c |= __shfl_down_sync(0xffffffffu, c, 2) << 8;
                c |= __shfl_down_sync(0xffffffffu, c, 4) << 16;
                if (in && (lane & 7) == 0) *reinterpret_cast<uint32_t*>(a.sf + scale_offset(a, r[b], h[b])) = c;
            } else if (in && (lane & 1) == 0) {
                a.sf[scale_offset(a, r[b], h[b])] = static_cast<uint8_t>(c);
            }
        }
    }
}

// A lane reads back one half: 8.5 bytes read and 32 written. 8192 x 8192: 31.5
// us, 5.4 TB/s (2 halves in flight 32.6, 4 blocks per SM 36.0).
__global__ void __launch_bounds__(THREADS, DEQUANT_PER_SM) dequant_kernel(const RowArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * THREADS;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i0 < a.total; i0 += BATCH * stride) {
        uint2 q[BATCH];
        uint32_t c[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t i = i0 + b * stride;
            if (i < a.total) {
                uint32_t h;
                const uint32_t r = divide(static_cast<uint32_t>(i), a.halves, a.inv, h);
                q[b] = *reinterpret_cast<const uint2*>(a.q + i * 8);
                c[b] = a.sf[scale_offset(a, r, h)];
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t i = i0 + b * stride;
            if (i < a.total) {
                const float s = e8m0_value(c[b]);
                uint4* y = reinterpret_cast<uint4*>(a.y) + 2 * i;
                const uint4 lo = e2m1x8_to_bf16(q[b].x, s), hi = e2m1x8_to_bf16(q[b].y, s);
                if (a.wide) {
                    store32(y, lo, hi);
                } else {
                    y[0] = lo;
                    y[1] = hi;
                }
            }
        }
    }
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

// Rows per launch: divide() takes fewer than 2^32 halves. Whole 128-row atoms.
constexpr int64_t MAX_HALVES = 0xF0000000ll;

// Calls launch(rows' arguments, blocks) for consecutive parts of the rows.
template <typename F>
int by_parts(const DeviceInfo& di, RowArgs a, int64_t R, int64_t rows, int64_t K, int64_t x_bytes, int batch, int per_sm,
             F&& launch) {
    a.halves = static_cast<uint32_t>(K / 16);
    a.inv = 0xFFFFFFFFu / a.halves;
    const int64_t part = MAX_HALVES / a.halves / 128 * 128;
    for (int64_t r0 = 0; r0 < rows; r0 += part) {
        const int64_t n = rows - r0 < part ? rows - r0 : part;
        RowArgs b = a;
        b.R = static_cast<uint32_t>(R - r0 < n ? (R > r0 ? R - r0 : 0) : n);
        b.total = n * b.halves;
        if (b.x) b.x = static_cast<const uint8_t*>(b.x) + r0 * b.ldx * x_bytes;
        b.q += r0 * (K / 2);
        b.sf += r0 * (K / 32);
        if (b.y) b.y += r0 * K;
        // as many blocks as are resident; fewer halves per thread while SMs would stay without
        int64_t blocks = (b.total + THREADS * batch - 1) / (THREADS * batch);
        if (blocks < di.num_sms) blocks = (b.total + THREADS - 1) / THREADS;
        if (blocks > static_cast<int64_t>(per_sm) * di.num_sms) blocks = static_cast<int64_t>(per_sm) * di.num_sms;
        if (int rc = launch(b, static_cast<unsigned>(blocks))) return rc;
    }
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
    RowArgs a{};
    a.x = x;
    a.q = q;
    a.sf = sf;
    a.ldx = ldx;
    a.tiled = tiled;
    a.groups = K % 128 == 0 && aligned(sf, 4);
    const bool bf16 = x_kind == METIS_A_BF16;
    a.wide = aligned(x, 32) && ldx * (bf16 ? 2 : 4) % 32 == 0;
    return by_parts(di, a, R, rows, K, bf16 ? 2 : 4, bf16 ? batch<__nv_bfloat16>() : batch<float>(), PER_SM, [&](const RowArgs& b, unsigned blocks) {
        return cuda_check(launch_pdl(bf16 ? quant_kernel<__nv_bfloat16> : quant_kernel<float>, dim3(blocks), dim3(THREADS),
                                     0, static_cast<cudaStream_t>(stream), 1, b),
                          "quant_mxfp4 launch");
    });
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
    RowArgs a{};
    a.q = const_cast<uint8_t*>(q);
    a.sf = const_cast<uint8_t*>(sf);
    a.y = static_cast<__nv_bfloat16*>(y_bf16);
    a.wide = aligned(y_bf16, 32);
    a.tiled = tiled;
    return by_parts(di, a, R, R, K, 0, BATCH, DEQUANT_PER_SM, [&](const RowArgs& b, unsigned blocks) {
        return cuda_check(launch_pdl(dequant_kernel, dim3(blocks), dim3(THREADS), 0, static_cast<cudaStream_t>(stream), 1, b),
                          "dequant_mxfp4 launch");
    });
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
    return launch_mxfp4_gemm(qa, sfa, (M + 127) / 128 * 128, qb, sfb, N, static_cast<__nv_bfloat16*>(y_bf16),
                             static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                             static_cast<cudaStream_t>(stream));
}
