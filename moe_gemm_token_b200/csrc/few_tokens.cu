// Default maths for few tokens with the weights read once: the routed-expert
// layer with FP8 or NVFP4 experts, and the NVFP4 weight-only product.
//   h[s] = W_up[e] x[t],  o[s] = W_down[e] h[s],  y[t] = bf16( sum_j w[t, j] o[t, j] )
// for the slots s = (t, j) with expert e = topk_ids[t, j]; FP32 sums, h and o
// kept in FP32. ("Lernex/Metis-1.6-Logos-FP8" and "-Praxis-NVFP4", "What
// --fast-math does": decoding for a few conversations widens the weights to 16
// bits as it multiplies, so that the weights are the only thing rounded.)
//
// The floor is the chosen experts' weights over HBM; what the kernels lose
// against it is the latency of the two dependent projections.
//
//  * few_kernel, one launch per projection. Each CTA builds the routing from
//    the ids itself: jobs (an expert with up to 8 or 16 of its slots), whose
//    16-row tiles are shared out evenly over the CTAs. A warp streams its
//    tiles' weights through lane-private places of shared memory (cp.async, any
//    row granularity: per-row bulk copies were bound by their issue, 46 per
//    microsecond and CTA; in flight per CTA, FP8 64 KB with 8 warps and 96 with
//    16, NVFP4 48 and 64 KB of codes), widens them to
//    FP16 (E4M3, and E2M1 times an E4M3 block scale, are exact FP16 values)
//    and multiplies with mma.sync m16n8k16, the weights as the 16 rows and the
//    job's tokens as the 8 columns. A tile's K is split over ks warps when
//    there are fewer tiles than warps; their sums meet in shared memory.
//  * The operand (x, then h) is staged as FP16 after a power-of-two shift of
//    its row: BF16 values keep all their bits within 2^-29 of the row's
//    largest. FP32 values become two FP16 values, the rounded one and the
//    rounded rest (22 significant bits, 2^-39 of the row's largest): two
//    columns of the MMA whose sums are added. One FP16 value alone would put
//    0.0009 (RMS) between the results and those of FP32 sums; two keep what
//    the FP32 sums give, and cost no MMA while a job has up to 4 slots.
//  * Few slots (h of all of them fits a CTA): the down-projection's CTAs own
//    output rows for every job and finish y themselves, two launches in all
//    (OWN). More: o goes through the workspace and combine_kernel (DOWN).
//  * The next kernel's prologue (routing, first weights) overlaps this one
//    through programmatic dependent launch, where an SM has room for both.
//
// Sums are added in a fixed order and no result depends on an atomic's order.
//
// With few weights per SM every instruction before the stream runs once, out
// of a cold instruction cache: the code there is kept short (loops not
// unrolled, tails left by `break` instead of predicated), which took a call of
// one token from 13.6 to 13.0 us (FP8) and from 12.7 to 12.1 (NVFP4).
#include <type_traits>

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

enum Mode { UP = 0, DOWN = 1, OWN = 2, DENSE = 3 };

// FP16 values that an operand element is staged as, each a row of its own.
template <int MODE>
constexpr int PARTS = MODE == DOWN || MODE == OWN ? 2 : 1;

// Geometry by warps per CTA: 8 warps leave room on an SM for a CTA of the next
// kernel, whose prologue then overlaps (few weights per SM: latency); 16 take
// an SM by themselves and share one staged operand (many weights per SM).
// DEPTH: pieces (2 KB) in flight per warp. 8 warps: OWN shares the SM with the
// up-projection, where both fit, and reads its pieces ahead while that one runs
// (us a call, OWN with 3, 4 and 5 pieces: FP8 1 token 2048 x 1024 13.1, 12.7,
// 12.6; 4 tokens top-4 2048 x 512 13.9, 13.5, 15.9, where 5 do not fit; 1 token
// 4096 x 1024 21.4, 19.4, 19.3; NVFP4 1 token 3 pieces 12.07, 4 pieces 12.17, 5
// pieces 14.6). 16 warps, us per
// call: FP8, 32 tokens 2 pieces 57.0, 3 pieces 56.4; NVFP4, which its
// widening instructions bound, 64 tokens 2 pieces 28.3, 3 pieces 29.2.
template <int FMT, int MODE, int GMAX, int W>
struct Cta {
    static constexpr int DEPTH = W == 8     ? (FMT == NVFP4 ? 3 : 4)
                                 : FMT == FP8 ? 3
                                              : 2;
};

// Per-format geometry. A piece is 16 rows by 128 bytes, in two halves: lane
// (g, t) = (lane / 4, lane % 4) holds bytes 16 t .. 16 t + 15 of each half of
// rows g and g + 8. (With pieces of 64 bytes the addresses and the loop cost
// a fifth of the instructions.)
template <int FMT>
struct Geo {
    static constexpr int EL = FMT == FP8 ? 64 : 128;     // elements of K per half
    static constexpr int CH = EL / 32;                   // 8-element chunks of K per lane and half
    // a piece in the ring: codes [half][row of the lane][32][16]; then words:
    // FP8 per lane the channel scales of its two rows; NVFP4 the block scales
    // [64-element chunk][16 rows][4], and per lane the global scale
    static constexpr int WORDS = 2048, GLOBAL = FMT == FP8 ? WORDS : WORDS + 256;
    static constexpr int SLOT = FMT == FP8 ? WORDS + 256 : GLOBAL + 128;
};

struct Args {
    const void* in;        // UP, DENSE: BF16 [tokens, K]; DOWN, OWN: FP32 [S, K]
    Weights w;
    const int32_t* ids;    // [S]; DENSE: null
    const float* tw;       // OWN: [S] routing weights
    int E, S, T, topk;     // DENSE: E = 1, S = T = tokens
    int P;                 // operand rows that are staged at a time, at most
    int by_token;          // UP: all tokens are staged, before the routing is known
    uint32_t grid_inv, tiles_inv;  // floor((2^32 - 1) / d) of the grid and of the tiles of a job
    int pitch;             // bytes between staged FP16 rows: 64 mod 128
    void* out;             // UP, DOWN: FP32 [S, N]; OWN: BF16 [T, N]; DENSE: BF16 [T, N]
    uint32_t* status;
};

// A tile of 16 rows against the columns of one pass, as the threads that add
// the warps' sums see it.
struct Item {
    int slot0, n, p, pe;   // first entry in the slot list, columns, first place, end of the places
};

// Bytes between staged operand rows: whole pieces, and 64 mod 128 so that the
// lanes of two rows read different banks.
template <int FMT>
constexpr int operand_pitch(int K) {
    return (K + 2 * Geo<FMT>::EL - 1) / (2 * Geo<FMT>::EL) * (2 * Geo<FMT>::EL) * 2 + 64;
}

// n / d and the rest, with inv = floor((2^32 - 1) / d): the product is at most one short.
__device__ __forceinline__ int divide(uint32_t n, uint32_t d, uint32_t inv, int& rest) {
    uint32_t q = __umulhi(n, inv), r = n - q * d;
    if (r >= d) ++q, r -= d;
    rest = static_cast<int>(r);
    return static_cast<int>(q);
}

// Shared memory: ring | partial sums | staged operand | its scales | items | routing | outputs.
struct Smem {
    int part, x, unshift, items, route, own, total;
};
template <int FMT, int MODE, int GMAX, int W>
__host__ __device__ inline Smem smem_layout(int slot_bytes, int P, int pitch, int E, int S) {
    constexpr bool routed = MODE != DENSE, own = MODE == OWN;
    Smem s;
    s.part = W * Cta<FMT, MODE, GMAX, W>::DEPTH * slot_bytes;
    s.x = s.part + (GMAX == 1 ? 2 : 1) * W * 512 * GMAX;
    s.unshift = s.x + P * PARTS<MODE> * pitch;
    s.items = s.unshift + ((P * 8 + 15) & ~15);
    s.route = s.items + 2 * W * static_cast<int>(sizeof(Item));
    s.own = s.route + (routed ? 4 * (E + 4 * S + 18) : 16);
    s.own = (s.own + 15) & ~15;
    s.total = s.own + (own ? S * 17 * 4 : 0);
    return s;
}

// Asynchronous copies to shared memory; `zero`: the source is not read and
// zeros are written.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool zero) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tcp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst),
                 "l"(src), "r"(static_cast<int>(zero)) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool zero) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tcp.async.ca.shared.global [%0], [%1], 4, p;\n\t}" ::"r"(dst),
                 "l"(src), "r"(static_cast<int>(zero)) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t p) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int DEPTH>
__device__ __forceinline__ void cp_async_wait_oldest() {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 bytes -> FP16 pairs (bytes 0, 1) and (2, 3), exactly.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
// Eight E2M1 codes -> four FP16 pairs in element order, exactly.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two FP32 values -> FP16, nearest even, infinities the largest finite value.
__device__ __forceinline__ uint32_t f16x2_saturated(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The two E4M3 scales in the low half of w, each as an FP16 pair of itself.
__device__ __forceinline__ void scale_pairs(uint32_t w, uint32_t& s0, uint32_t& s1) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
    s0 = __byte_perm(h, h, 0x1010);
    s1 = __byte_perm(h, h, 0x3232);
}

// Row of the matrix that stands at place p of its expert: the NVFP4 rows are
// taken in the order of the tiled scales, so that neighbouring places have
// neighbouring scale bytes.
template <int FMT>
__device__ __forceinline__ int place_to_row(int p) {
    return FMT == FP8 ? p : (p & ~127) | ((p & 3) << 5) | ((p & 127) >> 2);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Operand rows [K] are staged as FP16 after the power-of-two shift that
// brings a row's largest magnitude into [2^14, 2^15) (exact for BF16 values
// within 2^-29 of the largest; FP32 values with PARTS = 2 lose less than 2^-22
// of theirs or 2^-39 of the largest). A row with an infinity or a NaN is
// shifted as if its largest were 2^128, so that its finite values stay finite
// (what they add to a sum with an infinity does not matter); with two parts the
// first is the largest FP16 value and the second the infinity. 16-byte chunks
// are stored in the order in which the lanes read them (operand_chunk), zeros
// from K to the end of the last piece.
template <int FMT>
__device__ __forceinline__ int operand_chunk(int q) {
    constexpr int C = Geo<FMT>::CH;  // a half's chunk t * C + i is stored at i * 4 + t
    const int piece = q / (4 * C), r = q % (4 * C);
    return piece * 4 * C + (r % C) * 4 + r / C;
}
// Staging n operand rows by all warps: row i is src(i) and its part j goes to
// dst + (PARTS * i + j) * pitch. W / n' warps share a row (n' = n rounded up to a power of two), so
// that a few rows are read with one round trip, and a lane keeps its chunks
// in registers between the two steps (largest magnitude, shift) when they fit.
// The largest magnitude of three, NaN if one of them is NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
template <typename In>
struct Chunk;  // eight elements as loaded
template <>
struct Chunk<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(u[i]);
            v[2 * i + 1] = bf16_hi(u[i]);
        }
    }
    // bits of the largest magnitude, as binary32
    __device__ __forceinline__ uint32_t amax() const {
        const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                    __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
        return max(m & 0xFFFF0000u, m << 16);
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ uint32_t amax() const {
        return __float_as_uint(max3(max3(max3(max3(0.0f, a.x, a.y), a.z, a.w), b.x, b.y), b.z, b.w));
    }
};
constexpr int STAGE_U = 4;  // chunks of a lane in flight

template <int W>
__device__ __forceinline__ int warps_per_row(int n) {
    int wpr = W;
#pragma unroll 1
    while (wpr > 1 && n * wpr > W) wpr >>= 1;
    return wpr;
}
// Whether every lane's chunks fit its registers (one row and one batch each).
template <int W>
__device__ __forceinline__ bool staged_from_registers(int n, int K) {
    const int wpr = warps_per_row<W>(n);
    return n * wpr <= W && K / 8 <= STAGE_U * 32 * wpr;
}
// The loads of a batch: chunks q, q + step, ...
template <typename In>
__device__ __forceinline__ void load_chunks(Chunk<In> (&v)[STAGE_U], const In* row, int q, int step, int chunks) {
#pragma unroll
    for (int u = 0; u < STAGE_U; ++u) {
        if (q + u * step >= chunks) break;
        v[u].load(row + 8 * (q + u * step));
    }
}
// Ends with the rows visible to all threads. WHOLE: nothing is loaded before,
// and a warp takes whole rows when its registers hold one, both steps of a row
// after one read of it (us a call: 5 tokens, odd, 14.3 -> 13.0, 2 tokens 20.2 ->
// 18.6, 1 token 12.8 -> 12.5). `loaded`: the caller has made the loads
// (staged_from_registers holds); `maxima`: and found each warp's largest
// magnitude, [n][W].
template <int FMT, int W, int PARTS, bool WHOLE, typename In, typename Src>
__device__ __forceinline__ void stage_rows(int n, int K, uint8_t* dst, int pitch, float* unshift, uint32_t* amax,
                                           Chunk<In> (&v)[STAGE_U], bool loaded, const uint32_t* maxima, Src&& src) {
    constexpr int PC = Geo<FMT>::EL / 4;  // chunks of a piece
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool whole = WHOLE && K / 8 <= 32 * STAGE_U;
    const int wpr = whole ? 1 : warps_per_row<W>(n);
    const int chunks = K / 8, padded = (chunks + PC - 1) / PC * PC;
    const int q0 = (warp & (wpr - 1)) * 32 + lane, step = 32 * wpr;
    const int lw = 31 - __clz(wpr);
    const bool keep = staged_from_registers<W>(n, K);
    if (!maxima && !whole) {
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += 32 * W) amax[i] = 0u;
        __syncthreads();
#pragma unroll 1
        for (int i = warp >> lw; i < n; i += W >> lw) {
            const In* row = src(i);
            uint32_t m = 0;
#pragma unroll 1
            for (int q = q0; q < chunks; q += STAGE_U * step) {
                if (!loaded) load_chunks(v, row, q, step, chunks);
#pragma unroll
                for (int u = 0; u < STAGE_U; ++u) {
                    if (q + u * step >= chunks) break;
                    m = max(m, v[u].amax());
                }
            }
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) atomicMax(amax + i, m);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int i = warp >> lw; i < n; i += W >> lw) {
        const In* row = src(i);
        uint32_t m;
        if (whole) {
            load_chunks(v, row, q0, step, chunks);
            m = 0;
#pragma unroll
            for (int u = 0; u < STAGE_U; ++u) {
                if (q0 + u * step >= chunks) break;
                m = max(m, v[u].amax());
            }
        } else {
            m = maxima ? (lane < wpr ? maxima[i * W + lane] : 0u) : amax[i];
        }
        m = __reduce_max_sync(0xffffffffu, m);
        // floor(log2(m)) = bits' exponent - 127 (not finite: 128); a subnormal m has its leading bit at 31 - clz
        const int lg = m >= 0x00800000u ? static_cast<int>(m >> 23) - 127 : 31 - __clz(m) - 149;
        const int sh = m == 0 ? 0 : 14 - lg;
        // 2^sh and 2^-sh may leave FP32's normal range: two factors
        const int sa = max(-100, min(100, sh));
        const float fa = pow2(sa), fb = pow2(sh - sa);
        if (q0 == 0) unshift[i] = pow2(-sa) * pow2(sa - sh);
#pragma unroll 1
        for (int q = q0; q < padded; q += STAGE_U * step) {
            if (!keep && !whole) load_chunks(v, row, q, step, chunks);
#pragma unroll
            for (int u = 0; u < STAGE_U; ++u) {
                const int c = q + u * step;
                if (c >= padded) break;
                float f[8];
                v[u].get(f);
                if (sa != sh) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] *= fb;
                }
#pragma unroll
                for (int j = 0; j < PARTS; ++j) {
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float lo = j ? f[2 * k] : f[2 * k] * fa, hi = j ? f[2 * k + 1] : f[2 * k + 1] * fa;
                        if (j + 1 < PARTS) {
                            h[k] = f16x2_saturated(lo, hi);
                            // what the rounding left, exactly
                            const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
                            f[2 * k] = lo - r.x;
                            f[2 * k + 1] = hi - r.y;
                        } else {
                            const __half2 p = __floats2half2_rn(lo, hi);
                            h[k] = *reinterpret_cast<const uint32_t*>(&p);
                        }
                    }
                    // past K: zeros (a second batch there is not what the lane kept)
                    *reinterpret_cast<uint4*>(dst + (PARTS * i + j) * pitch + 16 * operand_chunk<FMT>(c)) =
                        c < chunks ? make_uint4(h[0], h[1], h[2], h[3]) : make_uint4(0, 0, 0, 0);
                }
            }
        }
    }
    __syncthreads();
}

// The work on the chosen experts as jobs: an expert with up to `columns` of its
// slots (the columns of one pass through its weights). An expert with more
// slots has several jobs, whose weights the L2 cache gives again.
struct Routing {
    int* expert;   // [jobs]
    int* start;    // [jobs + 1] first entry of each in slots
    int* slots;    // [S] by expert
    int* row;      // [S] the slot's operand row: its token (UP) or itself
    int jobs;
};

// Built by every CTA from the ids. Up to 32 slots: one warp, by matching ids
// (8 warps: first_id is the lane's);
// more: counts in shared memory and a scan over the experts. The order of a
// job's slots does not matter to the results (a slot is a column of the MMA),
// but which slots make a job has to be the same for all CTAs: where an expert
// has several jobs, its slots are put in ascending order.
template <int MODE, int THREADS>
__device__ __forceinline__ Routing build_routing(const Args& a, uint8_t* mem, int columns, int first_id) {
    int* count = reinterpret_cast<int*>(mem);                 // [E], then first entries
    Routing r;
    r.expert = count + a.E;
    r.start = r.expert + a.S;
    r.slots = r.start + a.S + 1;
    r.row = r.slots + a.S;
    int* jobs = r.row + a.S;
    const int lane = threadIdx.x % 32;
    // `c` slots of expert e, from entry `first` on: lane by lane one more set of jobs
    auto emit = [&](int e, int c, int first, int at) {
#pragma unroll 1
        for (int k = 0; k < c; k += columns, ++at) {
            r.expert[at] = e;
            r.start[at] = first + k;
        }
    };
    auto scan = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    if (a.S <= 32) {
        if (threadIdx.x < 32) {
            int e = THREADS == 256 ? first_id : lane < a.S ? a.ids[lane] : -1;
            const bool in = e >= 0 && e < a.E;
            if (lane < a.S && !in && blockIdx.x == 0) atomicOr(a.status, kDevErrBadIndex);
            if (!in) e = -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int lead = __ffs(same) - 1;
            const int c = in && lead == lane ? __popc(same) : 0;
            // slots in the low half, jobs in the high half
            const int own = c | ((c + columns - 1) / columns) << 16;
            const int incl = scan(own);
            emit(e, c, (incl - own) & 0xFFFF, (incl - own) >> 16);
            const int first = __shfl_sync(0xffffffffu, (incl - own) & 0xFFFF, lead);
            if (in) {
                const int at = first + __popc(same & ((1u << lane) - 1u));
                r.slots[at] = lane;
                r.row[at] = MODE == UP ? lane / a.topk : lane;
            }
            if (lane == 31) {
                r.start[incl >> 16] = incl & 0xFFFF;
                *jobs = incl >> 16;
            }
        }
        __syncthreads();
        r.jobs = *jobs;
        return r;
    }
    constexpr int SLOTS = MAX_S / THREADS, EXPERTS = MAX_E / THREADS;  // per thread
    int id[SLOTS], rank[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        const int s = threadIdx.x + i * THREADS;
        id[i] = s < a.S ? a.ids[s] : -1;
    }
    for (int e = threadIdx.x; e < a.E; e += THREADS) count[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        rank[i] = 0;
        if (id[i] >= 0 && id[i] < a.E) {
            rank[i] = atomicAdd(&count[id[i]], 1);
        } else {
            if (static_cast<int>(threadIdx.x) + i * THREADS < a.S && blockIdx.x == 0) atomicOr(a.status, kDevErrBadIndex);
            id[i] = -1;
        }
    }
    __syncthreads();
    // scan over the experts, EXPERTS consecutive ones per thread: slots in the
    // low half, jobs in the high half
    const int e0 = threadIdx.x * EXPERTS;
    int c[EXPERTS], own = 0;
    bool split = false;  // an expert with several jobs
#pragma unroll
    for (int k = 0; k < EXPERTS; ++k) {
        c[k] = e0 + k < a.E ? count[e0 + k] : 0;
        own += c[k] | ((c[k] + columns - 1) / columns) << 16;
        split |= c[k] > columns;
    }
    int incl = scan(own);
    if (lane == 31) jobs[threadIdx.x / 32] = incl;
    __syncthreads();
    {
        const int w = threadIdx.x / 32;
        incl += __reduce_add_sync(0xffffffffu, lane < w ? jobs[lane] : 0);
    }
    int first = (incl - own) & 0xFFFF, at = (incl - own) >> 16;
#pragma unroll
    for (int k = 0; k < EXPERTS; ++k) {
        if (c[k] > 0) {
            emit(e0 + k, c[k], first, at);
            count[e0 + k] = first | c[k] << 16;  // first entry, slots
            first += c[k];
            at += (c[k] + columns - 1) / columns;
        }
    }
    if (threadIdx.x == THREADS - 1) {
        r.start[incl >> 16] = incl & 0xFFFF;
        jobs[THREADS / 32] = incl >> 16;
    }
    if (__syncthreads_or(split)) {
        // an expert's slots in ascending order
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (id[i] >= 0) r.row[(count[id[i]] & 0xFFFF) + rank[i]] = threadIdx.x + i * THREADS;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (id[i] >= 0) {
                const int n = count[id[i]] >> 16, s = threadIdx.x + i * THREADS;
                const int* list = r.row + (count[id[i]] & 0xFFFF);
                if (n > columns) {
                    int below = 0;
                    for (int k = 0; k < n; ++k) below += list[k] < s;
                    rank[i] = below;
                }
            }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
        if (id[i] >= 0) {
            const int s = threadIdx.x + i * THREADS, to = (count[id[i]] & 0xFFFF) + rank[i];
            r.slots[to] = s;
            r.row[to] = MODE == UP ? s / a.topk : s;
        }
    r.jobs = jobs[THREADS / 32];
    __syncthreads();
    return r;
}

template <int FMT, int MODE, int GMAX, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) few_kernel(const Args a) {
    using G = Geo<FMT>;
    constexpr int THREADS = WARPS * 32, DEPTH = Cta<FMT, MODE, GMAX, WARPS>::DEPTH;
    constexpr int LOG = WARPS == 8 ? 3 : 4;
    // groups of 8 MMA columns in a pass, slots per group, and sums per lane and group
    constexpr int PT = PARTS<MODE>, GROUPS = GMAX * PT, SLOTS = 8 / PT, SUMS = 4 / PT;
    using In = typename std::conditional<MODE == UP || MODE == DENSE, __nv_bfloat16, float>::type;
    extern __shared__ __align__(128) uint8_t smem[];
    const Smem L = smem_layout<FMT, MODE, GMAX, WARPS>(G::SLOT, a.P, a.pitch, a.E, a.S);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane >> 2, t = lane & 3;
    const int N = a.w.N, K = a.w.K;
    const int row_bytes = FMT == FP8 ? K : K / 2;
    const int kp = (row_bytes + 127) / 128;  // pieces per tile of rows
    uint8_t* xs = smem + L.x;
    float* unshift = reinterpret_cast<float*>(smem + L.unshift);
    uint32_t* amax = reinterpret_cast<uint32_t*>(unshift + a.P);
    Item* items = reinterpret_cast<Item*>(smem + L.items);
    const In* in = static_cast<const In*>(a.in);

    // UP, DENSE: the ids or the operand may be the previous kernel's output.
    // DOWN, OWN: only the up-projection can still be running (it lets this
    // grid start after its own wait), so the routing and the weights may be
    // read before the wait, h not.
    if constexpr (MODE == UP || MODE == DENSE) {
        grid_dependency_wait();
        if (MODE == DENSE || WARPS != 8) grid_launch_dependents();
    }
    // The operand's loads are made early, before the weights fill the memory
    // system's queues: all tokens (by_token) before the routing, else the first
    // group's rows after it.
    Chunk<In> early[STAGE_U];
    bool loaded = false;
    auto load_early = [&](int n, auto&& src) {
        loaded = staged_from_registers<WARPS>(n, K);
        if (loaded) {
            const int wpr = warps_per_row<WARPS>(n), i = warp / wpr;
            if (i < n) load_chunks(early, src(i), (warp % wpr) * 32 + lane, 32 * wpr, K / 8);
        }
    };
    const bool by_token = MODE == UP && a.by_token;
    int first_id = -1;
    if (MODE != DENSE && WARPS == 8 && a.S <= 32 && lane < a.S) first_id = a.ids[lane];
    const uint32_t* maxima = nullptr;
    if (by_token) {
        load_early(a.T, [&](int i) { return in + static_cast<int64_t>(i) * K; });
        if (WARPS == 8 && loaded && a.S <= 32) {
            // the largest magnitudes while one warp waits for the ids (a call of one
            // token: FP8 13.0, 12.8 us; NVFP4 12.2, 11.9)
            uint32_t* to = reinterpret_cast<uint32_t*>(smem + L.part);
            const int wpr = warps_per_row<WARPS>(a.T), i = warp / wpr;
            if (i < a.T) {
                uint32_t m = 0;
#pragma unroll
                for (int u = 0; u < STAGE_U; ++u) {
                    if ((warp % wpr + u * wpr) * 32 + lane >= K / 8) break;
                    m = max(m, early[u].amax());
                }
                m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) to[i * WARPS + warp % wpr] = m;
            }
            maxima = to;
        }
    }

    const int columns = by_token ? 8 * GMAX : min(a.P, 8 * GMAX);  // of a job
    Routing rt{};
    if constexpr (MODE == DENSE) rt.jobs = (a.S + columns - 1) / columns;
    else rt = build_routing<MODE, THREADS>(a, smem + L.route, columns, first_id);
    auto job_expert = [&](int j) { return MODE == DENSE ? 0 : rt.expert[j]; };
    auto job_start = [&](int j) { return MODE == DENSE ? min(j * columns, a.S) : rt.start[j]; };

    // The share of this CTA. UP, DOWN, DENSE: tiles of 16 rows, of one job
    // after another: tile f of the share is tile (u0 + f) % job_tiles of job
    // (u0 + f) / job_tiles. OWN: rows of the output, in tiles of 16, each for
    // every job: tile f is job f % jobs of rows 16 (f / jobs) of the share.
    const int job_tiles = (N + 15) >> 4;
    int spare;
    const int each = divide(MODE == OWN ? N : rt.jobs * job_tiles, gridDim.x, a.grid_inv, spare);
    const int u0 = each * static_cast<int>(blockIdx.x) + min(static_cast<int>(blockIdx.x), spare);
    const int share = each + (static_cast<int>(blockIdx.x) < spare ? 1 : 0);
    const int total = MODE == OWN ? ((share + 15) >> 4) * rt.jobs : share;
    auto tile_job = [&](int f, int& tile) { return divide(u0 + f, job_tiles, a.tiles_inv, tile); };
    // Tiles are taken in groups whose operand rows are staged together: whole
    // jobs, as many as fit, shared out to the warps without a barrier. by_token:
    // one group; OWN: a group is 16 rows, the operand is staged for all of them.
    auto group_end = [&](int f) {
        if (MODE == OWN) return f + rt.jobs;
        if (by_token) return share;
        int tile, j = tile_job(f, tile);
        const int most = job_start(j) + a.P;
        ++j;
#pragma unroll 1
        while (j * job_tiles < u0 + share && job_start(j + 1) <= most) ++j;
        return min(j * job_tiles - u0, share);
    };

    // ks warps share a tile's K, so that WARPS / ks teams work on tiles of
    // their own: the split with the fewest pieces in a row, the joining of a
    // round's sums counted as one piece (a tile per warp needs none).
    int ks = 1, lt = LOG;  // teams = 1 << lt
    {
        const int tiles = MODE == OWN ? rt.jobs : share;
        int best = 0x7fffffff;
#pragma unroll
        for (int l = 0; l <= LOG; ++l) {
            const int k = WARPS >> l;
            const int cost = ((tiles + (1 << l) - 1) >> l) * (((kp + k - 1) >> (LOG - l)) + (k > 1 ? 1 : 0));
            if (cost < best) best = cost, ks = k, lt = l;
        }
    }
    const int teams = 1 << lt, team = warp >> (LOG - lt), kslice = warp & (ks - 1);

    // ---- weight stream: this warp's pieces in order, DEPTH of them in flight
    // in lane-private places of the ring (a lane reads back what it copied; of
    // the NVFP4 block scales, what the warp copied).
    // Rows past the tile's end repeat its first row (their sums are not
    // stored); bytes past the end of a row are zeros.
    const int pieces = kslice < kp ? (kp - kslice + ks - 1) >> (LOG - lt) : 0;  // of a tile, for this warp
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * DEPTH * G::SLOT);
    int rf = team - teams, rend = 0, rleft = 0, rrem = 0, srem = 0;  // tile to request, end of its group
    int rrow = u0 - 16;                                    // OWN: first row of the group
    const uint8_t *wp0 = nullptr, *wp1 = nullptr, *sp = nullptr;
    auto next_tile = [&](uint32_t place) {
        rf += teams;
#pragma unroll 1
        while (rf >= rend) {
            if (rend >= total) {
                rf = rend = total;
                return;
            }
            rf = rend + team;
            rend = group_end(rend);
            if (MODE == OWN) rrow += 16;
        }
        int tile = 0;
        const int j = MODE == OWN ? rf - rend + rt.jobs : tile_job(rf, tile);
        const int e = job_expert(j);
        const int pb = MODE == OWN ? rrow : 16 * tile, p = pb + g, pe = MODE == OWN ? u0 + share : N;
        const uint32_t row0 = static_cast<uint32_t>(e * N + place_to_row<FMT>(p < pe ? p : pb));
        const uint32_t row1 = static_cast<uint32_t>(e * N + place_to_row<FMT>(p + 8 < pe ? p + 8 : pb));
        const int at = 128 * kslice + 16 * t;
        wp0 = a.w.q + static_cast<uint64_t>(row0) * static_cast<uint32_t>(row_bytes) + at;
        wp1 = a.w.q + static_cast<uint64_t>(row1) * static_cast<uint32_t>(row_bytes) + at;
        rrem = row_bytes - at;
        rleft = pieces;
        if constexpr (FMT == FP8) {
            cp_async4(place + G::WORDS + 4 * lane, a.w.s + row0, false);
            cp_async4(place + G::WORDS + 128 + 4 * lane, a.w.s + row1, false);
        } else {
            // the places' scale words of a chunk are consecutive. 16 places from a
            // multiple of 16 on (all but OWN): 16 bytes by lane, four chunks of
            // K; OWN: word by word, two chunks
            const int pl = MODE == OWN ? min(pb + (lane & 15), pe - 1) : pb + 4 * (lane & 3);
            const int chunk = 4 * kslice + (MODE == OWN ? lane >> 4 : lane >> 2);
            sp = a.w.sf + static_cast<uint64_t>((static_cast<uint32_t>(e * N + pl) >> 7) * (K / 64) + chunk) * 512 + 4 * (pl & 127);
            srem = K / 64 - chunk;
            cp_async4(place + G::GLOBAL + 4 * lane, a.w.s + e, false);
        }
    };
    auto request = [&](uint32_t to) {
        if (rleft == 0 && rf < total) next_tile(to);
        if (rleft > 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool past = rrem <= 64 * h;
                cp_async16(to + 1024 * h + 16 * lane, wp0 + 64 * h, past);
                cp_async16(to + 1024 * h + 512 + 16 * lane, wp1 + 64 * h, past);
            }
            wp0 += 128 * ks;
            wp1 += 128 * ks;
            rrem -= 128 * ks;
            if constexpr (FMT == NVFP4) {
                if constexpr (MODE == OWN) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        cp_async4(to + G::WORDS + 128 * h + 4 * lane, sp + 1024 * h, srem <= 2 * h);
                } else if (lane < 16) {
                    cp_async16(to + G::WORDS + 16 * lane, sp, srem <= 0);
                }
                sp += 2048 * ks;
                srem -= 4 * ks;
            }
            --rleft;
        }
        cp_async_commit();
    };
    if (pieces == 0) rf = rend = total;
    // the first group's operand rows, in the order of the slot list
    if constexpr (MODE == UP || MODE == DENSE) {
        if (!by_token && total > 0) {
            int tile;
            const int base = job_start(tile_job(0, tile)), n = job_start(tile_job(group_end(0) - 1, tile) + 1) - base;
            load_early(n, [&](int i) { return in + static_cast<int64_t>(MODE == DENSE ? base + i : rt.row[base + i]) * K; });
        }
    }
    // UP beside whose CTAs the next kernel's find room: they start when the
    // operand is staged, so that their first copies do not hold up this
    // kernel's, unless there is little to stream after that (us a call, started
    // at once and late: FP8 1 token 14.0, 13.5; 1024 x 512, top-4 9.9, 10.5).
    const bool late = MODE == UP && WARPS == 8 && 2 * total * kp > WARPS * DEPTH;
    if (MODE == UP && WARPS == 8 && !late) grid_launch_dependents();
    // fill the ring
#pragma unroll 1
    for (int d = 0; d < DEPTH; ++d) request(ring + d * G::SLOT);
    uint32_t place = ring;  // of the oldest piece

    // OWN: outputs per slot and row of 16; the slots' routing weights behind them
    float* own = reinterpret_cast<float*>(smem + L.own);
    if constexpr (MODE == OWN) {
#pragma unroll 1
        for (int s = threadIdx.x; s < a.S; s += THREADS) {
            const int id = a.ids[s];
            own[a.S * 16 + s] = a.tw[s];
            // outputs of a slot without an expert stay zero, and so does its weight
            if (id < 0 || id >= a.E) {
                own[a.S * 16 + s] = 0.0f;
#pragma unroll 1
                for (int i = 0; i < 16; ++i) own[s * 16 + i] = 0.0f;
            }
        }
    }
    if constexpr (MODE == DOWN || MODE == OWN) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    int buf = 0;
    for (int f0 = 0, f1; f0 < total; f0 = f1) {
        f1 = group_end(f0);
        // ---- operand rows, in the order of the slot list (OWN: those of slots
        // without an expert are not in it), or the tokens
        int base = 0, unused;
        if (MODE != OWN && !by_token) base = job_start(tile_job(f0, unused));
        if (!(MODE == OWN || by_token) || f0 == 0) {
            if (f0 > 0) __syncthreads();
            const int n = by_token ? a.T : job_start(MODE == OWN ? rt.jobs : tile_job(f1 - 1, unused) + 1) - base;
            stage_rows<FMT, WARPS, PT, MODE == DOWN || MODE == OWN, In>(n, K, xs, a.pitch, unshift, amax, early, loaded, maxima, [&](int i) {
                return in + static_cast<int64_t>(by_token ? i : MODE == DENSE ? base + i : rt.row[base + i]) * K;
            });
            loaded = false;
            if (late && f0 == 0) grid_launch_dependents();
        }
        const int own_row = MODE == OWN ? 16 * (f0 / max(rt.jobs, 1)) : 0;  // of the share
        for (int fr = f0; fr < f1; fr += teams) {
            const bool mine = fr + team < f1;
            // one group of columns (GMAX = 1): two chains of MMAs, added at the end
            constexpr int ACCS = GROUPS == 1 ? 2 : GROUPS;
            float acc[ACCS][4];
#pragma unroll
            for (int q = 0; q < ACCS; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.0f;
            int start = 0, n = 0, p0 = u0 + own_row;
            const int pe = MODE == OWN ? u0 + share : N;
            if (mine) {
                int tile = 0;
                const int j = MODE == OWN ? fr + team - f0 : tile_job(fr + team, tile);
                if (MODE != OWN) p0 = 16 * tile;
                start = job_start(j);
                n = job_start(j + 1) - start;
                // staged row of the job's slot c; slots past n repeat the first one: their
                // sums are not stored. MMA column g of group q is part g % PT of slot SLOTS q + g / PT.
                auto column = [&](int c) {
                    const int at = start + (c < n ? c : 0);
                    return by_token ? rt.row[at] : at - base;
                };
                uint32_t xp[GROUPS];
#pragma unroll
                for (int q = 0; q < GROUPS; ++q)
                    xp[q] = smem_u32(xs) + (column(SLOTS * q + g / PT) * PT + g % PT) * a.pitch + kslice * (4 * G::EL) + 16 * t;
                float sr[2] = {0.0f, 0.0f};
                if (pieces > 0) {
                    cp_async_wait_oldest<DEPTH>();
                    sr[0] = __uint_as_float(ld_shared4(place + G::GLOBAL + 4 * lane));
                    sr[1] = FMT == FP8 ? __uint_as_float(ld_shared4(place + G::WORDS + 128 + 4 * lane)) : sr[0];
                }
                auto run = [&](auto groups) {
                    constexpr int NG = decltype(groups)::value, SECOND = GMAX == 1 && NG == 1 ? 1 : 0;
#pragma unroll 1
                    for (int i = 0; i < pieces; ++i) {
                        cp_async_wait_oldest<DEPTH>();
                        if constexpr (FMT == NVFP4) __syncwarp();  // the scales are other lanes' copies
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 wa = ld_shared16(place + 1024 * h + 16 * lane);
                            const uint4 wb = ld_shared16(place + 1024 * h + 512 + 16 * lane);
                            uint32_t fa[2] = {0, 0}, fb[2] = {0, 0};
                            if constexpr (FMT == NVFP4) {
                                const uint32_t words = place + G::WORDS + 64 * (2 * h + (t >> 1)) + 4 * g;
                                scale_pairs(ld_shared4(words) >> (16 * (t & 1)), fa[0], fa[1]);
                                scale_pairs(ld_shared4(words + 32) >> (16 * (t & 1)), fb[0], fb[1]);
                            }
                            const uint32_t va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
                            // a chunk of 8 elements of K per lane at a time: rows g and g + 8 as the A
                            // operand of two MMAs (4 elements of K each), every group of 8 columns
#pragma unroll
                            for (int c = 0; c < G::CH; ++c) {
                                uint32_t A[2][4];
                                if constexpr (FMT == FP8) {
#pragma unroll
                                    for (int j = 0; j < 2; ++j) {
                                        e4m3x4_to_f16(va[2 * c + j], A[j][0], A[j][2]);
                                        e4m3x4_to_f16(vb[2 * c + j], A[j][1], A[j][3]);
                                    }
                                } else {
                                    uint32_t ha[4], hb[4];
                                    e2m1x8_to_f16(va[c], ha);
                                    e2m1x8_to_f16(vb[c], hb);
#pragma unroll
                                    for (int j = 0; j < 2; ++j) {
                                        A[j][0] = mul_f16x2(ha[2 * j], fa[c / 2]);
                                        A[j][2] = mul_f16x2(ha[2 * j + 1], fa[c / 2]);
                                        A[j][1] = mul_f16x2(hb[2 * j], fb[c / 2]);
                                        A[j][3] = mul_f16x2(hb[2 * j + 1], fb[c / 2]);
                                    }
                                }
#pragma unroll
                                for (int q = 0; q < NG; ++q) {
                                    const uint4 xv = ld_shared16(xp[q] + 2 * G::EL * h + 64 * c);
                                    mma_16816(acc[q], A[0][0], A[0][1], A[0][2], A[0][3], xv.x, xv.y);
                                    mma_16816(acc[SECOND + q], A[1][0], A[1][1], A[1][2], A[1][3], xv.z, xv.w);
                                }
                            }
                        }
#pragma unroll
                        for (int q = 0; q < NG; ++q) xp[q] += ks * (4 * G::EL);
                        if constexpr (FMT == NVFP4) __syncwarp();  // all lanes have read them
                        request(place);
                        place = place == ring + (DEPTH - 1) * G::SLOT ? ring : place + G::SLOT;
                    }
                    if constexpr (SECOND) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[0][j] += acc[1][j], acc[1][j] = 0.0f;
                    }
                };
                constexpr int LESS = GROUPS > 1 ? GROUPS / 2 : 1;  // groups of a job with few slots
                if (GROUPS == 1 || n <= LESS * SLOTS) run(std::integral_constant<int, LESS>());
                else run(std::integral_constant<int, GROUPS>());
                // the parts' sums, then the scales: of the rows, and of the columns' operand rows
                // (last: the sum of a token near FP32's largest, shifted back, may not be an FP32 value yet)
#pragma unroll
                for (int q = 0; q < GROUPS; ++q) {
                    if constexpr (PT == 2) acc[q][0] += acc[q][1], acc[q][1] = acc[q][2] + acc[q][3];
#pragma unroll
                    for (int j = 0; j < SUMS / 2; ++j) {
                        const float u = unshift[column(SLOTS * q + SUMS / 2 * t + j)];
                        acc[q][j] = acc[q][j] * sr[0] * u;
                        acc[q][SUMS / 2 + j] = acc[q][SUMS / 2 + j] * sr[1] * u;
                    }
                }
            }
            // slot and place of sum j of a lane (g, t) and group q: SUMS / 2 slots of row g, then of row g + 8
            auto slot_of = [](int q, int t, int j) { return SLOTS * q + SUMS / 2 * t + j % (SUMS / 2); };
            auto place_of = [](int p, int g, int j) { return p + g + 8 * (j / (SUMS / 2)); };
            // value v of column c of the job whose slots start at `at`, at place p
            auto put = [&](int at, int c, int p, float v) {
                const int row = place_to_row<FMT>(p);
                if constexpr (MODE == DENSE) {
                    static_cast<__nv_bfloat16*>(a.out)[static_cast<int64_t>(at + c) * N + row] = __float2bfloat16_rn(v);
                } else {
                    const int sl = rt.slots[at + c];
                    if constexpr (MODE == OWN) own[sl * 16 + (p - u0 - own_row)] = v;
                    else static_cast<float*>(a.out)[static_cast<int64_t>(sl) * N + row] = v;
                }
            };
            if (ks == 1) {
                if (mine) {
#pragma unroll
                    for (int q = 0; q < GROUPS; ++q)
#pragma unroll
                        for (int j = 0; j < SUMS; ++j) {
                            const int c = slot_of(q, t, j), p = place_of(p0, g, j);
                            if (c < n && p < pe) put(start, c, p, acc[q][j]);
                        }
                }
            } else {
                // ---- the warps' sums meet in shared memory, added in a fixed order
                float* part = reinterpret_cast<float*>(smem + L.part) + buf * (WARPS * 128 * GMAX);
                if (mine) {
#pragma unroll
                    for (int q = 0; q < GROUPS; ++q)
                        if (SLOTS * q < n) {
                            float* to = part + (warp * GROUPS + q) * (32 * SUMS) + SUMS * lane;
                            if constexpr (PT == 2) *reinterpret_cast<float2*>(to) = make_float2(acc[q][0], acc[q][1]);
                            else *reinterpret_cast<float4*>(to) = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
                        }
                }
                if (kslice == 0 && lane == 0) items[buf * WARPS + team] = Item{start, mine ? n : 0, p0, pe};
                __syncthreads();
                for (int o = threadIdx.x; o < teams * GMAX * 128; o += THREADS) {
                    const int tm = o / (GMAX * 128), q = o / (32 * SUMS) % GROUPS, at = o % (32 * SUMS);
                    const Item it = items[buf * WARPS + tm];
                    const int l = at / SUMS, c = slot_of(q, l & 3, at % SUMS), p = place_of(it.p, l >> 2, at % SUMS);
                    if (c >= it.n || p >= it.pe) continue;
                    float sum = 0.0f;
                    for (int w = 0; w < ks; ++w) sum += part[((tm * ks + w) * GROUPS + q) * (32 * SUMS) + at];
                    put(it.slot0, c, p, sum);
                }
                if constexpr (GMAX == 1) buf ^= 1;
                else __syncthreads();  // one buffer
            }
        }
        if constexpr (MODE == OWN) {
            // every job has given its part of these 16 rows
            __syncthreads();
            for (int i = threadIdx.x; i < a.T * 16; i += THREADS) {
                const int tk = i >> 4, p = u0 + own_row + (i & 15);
                if (p >= u0 + share) continue;
                float y = 0.0f;
                for (int sl = tk * a.topk; sl < (tk + 1) * a.topk; ++sl) y = fmaf(own[a.S * 16 + sl], own[sl * 16 + (i & 15)], y);
                static_cast<__nv_bfloat16*>(a.out)[static_cast<int64_t>(tk) * N + place_to_row<FMT>(p)] = __float2bfloat16_rn(y);
            }
            __syncthreads();
        }
    }
    if constexpr (MODE == OWN) {
        if (rt.jobs == 0) {  // no token has an expert
            for (int i = static_cast<int>(blockIdx.x) * THREADS + threadIdx.x; i < a.T * N;
                 i += static_cast<int>(gridDim.x) * THREADS)
                static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(0.0f);
        }
    }
}

// y[t] = bf16( sum_j w[t, j] o[t, j] ), FP32, j ascending; slots of no expert
// add nothing. A thread makes four columns of one token, COMBINE_U slots'
// values in flight.
constexpr int COMBINE_U = 8;
__global__ void __launch_bounds__(128) combine_kernel(const float* __restrict__ o, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ tw, int topk, int E, int H,
                                                      __nv_bfloat16* __restrict__ y) {
    const int n = 4 * (blockIdx.x * 128 + threadIdx.x);
    const int t = blockIdx.y;
    grid_dependency_wait();
    grid_launch_dependents();
    if (n >= H) return;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < topk; j0 += COMBINE_U) {
        float4 v[COMBINE_U];
        float w[COMBINE_U];
        bool in[COMBINE_U];
#pragma unroll
        for (int u = 0; u < COMBINE_U; ++u) {
            const int s = t * topk + j0 + u;
            in[u] = false;
            if (j0 + u < topk) {
                const int e = ids[s];
                w[u] = tw[s];
                // (an id of no expert: o was not written there, and is not used)
                v[u] = *reinterpret_cast<const float4*>(o + static_cast<int64_t>(s) * H + n);
                in[u] = e >= 0 && e < E;
            }
        }
#pragma unroll
        for (int u = 0; u < COMBINE_U; ++u)
            if (in[u]) {
                acc[0] = fmaf(w[u], v[u].x, acc[0]);
                acc[1] = fmaf(w[u], v[u].y, acc[1]);
                acc[2] = fmaf(w[u], v[u].z, acc[2]);
                acc[3] = fmaf(w[u], v[u].w, acc[3]);
            }
    }
    *reinterpret_cast<uint2*>(y + static_cast<int64_t>(t) * H + n) =
        make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
}

// NVFP4 weights [N, K] widened exactly to BF16, D2(q) D(sf) (six significant
// bits), and the global scale repeated for every column of the product. One
// lane per block of 16: 8.5 bytes read, 32 written (HBM-bound, mostly into L2).
constexpr int WIDEN_BATCH = 4;
__global__ void __launch_bounds__(256) widen_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sf,
                                                    const float* __restrict__ g, uint32_t blocks, uint32_t row_blocks,
                                                    uint32_t inv, int N, uint4* __restrict__ out, float* __restrict__ col) {
    // the workspace may still be read by the previous kernel
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t stride = gridDim.x * 256u, i0 = blockIdx.x * 256u + threadIdx.x;
    for (uint32_t n = i0; n < static_cast<uint32_t>(N); n += stride) col[n] = *g;
    for (uint64_t base = i0; base < blocks; base += static_cast<uint64_t>(WIDEN_BATCH) * stride) {
        uint2 w[WIDEN_BATCH];
        uint32_t c[WIDEN_BATCH];
#pragma unroll
        for (int u = 0; u < WIDEN_BATCH; ++u) {
            const uint64_t i = base + static_cast<uint64_t>(u) * stride;
            if (i < blocks) {
                int b;
                const uint32_t r = divide(static_cast<uint32_t>(i), row_blocks, inv, b);
                w[u] = __ldg(reinterpret_cast<const uint2*>(q) + i);
                c[u] = __ldg(sf + static_cast<uint64_t>((r >> 7) * (row_blocks >> 2) + (b >> 2)) * 512 + 16 * (r & 31) +
                             4 * ((r & 127) >> 5) + (b & 3));
            }
        }
#pragma unroll
        for (int u = 0; u < WIDEN_BATCH; ++u) {
            const uint64_t i = base + static_cast<uint64_t>(u) * stride;
            if (i >= blocks) continue;
            uint32_t s, unused;
            scale_pairs(c[u], s, unused);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t h[4], o[4];
                e2m1x8_to_f16(k ? w[u].y : w[u].x, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t v = mul_f16x2(h[j], s);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
                    o[j] = pack_bf16x2(f.x, f.y);
                }
                out[2 * i + k] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
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

// The shared memory of few_kernel with P staged operand rows (a.pitch is set).
template <int FMT, int MODE, int GMAX, int W>
int few_bytes(const Args& a, int P) {
    return smem_layout<FMT, MODE, GMAX, W>(Geo<FMT>::SLOT, P, a.pitch, a.E, a.S).total;
}

// Sets the operand's layout: as many staged rows P as are of use (OWN: all
// slots; by_token: all tokens; else the slots of two jobs) and fit: for 8 warps
// in half of the shared memory if that holds a job's rows, so that the next
// kernel's CTAs find room, else in all of it. False: not even one does, or not
// all where all are needed.
template <int FMT, int MODE, int GMAX, int W>
bool stage_plan(const DeviceInfo& di, Args& a) {
    a.pitch = operand_pitch<FMT>(a.w.K);
    const int base = few_bytes<FMT, MODE, GMAX, W>(a, 0) + 32;  // rounding
    const int row = PARTS<MODE> * a.pitch + 8;
    const int half = (112 * 1024 - base) / row, full = (di.max_smem_optin - base) / row;
    const int per_job = a.T < 8 * GMAX ? a.T : 8 * GMAX;
    // a few tokens that all threads read with one round trip
    a.by_token = MODE == UP && a.T <= W && static_cast<int64_t>(a.T) * a.w.K <= 8 * STAGE_U * 32 * W;
    const int want = a.by_token ? a.T : MODE == OWN || a.S < 2 * per_job ? a.S : 2 * per_job;
    const int room = W == 8 && half >= (MODE == OWN ? want : per_job) ? half : full;
    a.P = want < room ? want : room;
    return a.P >= 1 && (a.P >= want || !(MODE == OWN || a.by_token));
}

// Launches few_kernel, one CTA per SM.
template <int FMT, int MODE, int GMAX, int W>
int launch_few(const DeviceInfo& di, Args a, cudaStream_t st) {
    static std::atomic<uint64_t> done[64];
    int rc = once_per_context(done, di.device, [&] {
        const auto f = few_kernel<FMT, MODE, GMAX, W>;
        int r = cuda_check(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, di.max_smem_optin),
                           "cudaFuncSetAttribute(few tokens)");
        // the whole carveout: an SM set up for less would not take the next
        // kernel's CTA beside this one's (FP8, one token: 16.5 -> 14.9 us a call)
        if (!r)
            r = cuda_check(cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                cudaSharedmemCarveoutMaxShared),
                           "cudaFuncSetAttribute(few tokens, carveout)");
        return r;
    });
    if (rc) return rc;
    if (!stage_plan<FMT, MODE, GMAX, W>(di, a))
        return fail(METIS_ERR_UNSUPPORTED, "few-token kernel: K=%d is too long", a.w.K);
    a.grid_inv = 0xFFFFFFFFu / static_cast<uint32_t>(di.num_sms);
    a.tiles_inv = 0xFFFFFFFFu / static_cast<uint32_t>((a.w.N + 15) / 16);
    return cuda_check(launch_pdl(few_kernel<FMT, MODE, GMAX, W>, dim3(di.num_sms), dim3(W * 32), few_bytes<FMT, MODE, GMAX, W>(a, a.P), st, 1, a),
                      "few-token kernel launch");
}

// By the columns that one pass multiplies (8 or 16), the weight bytes that
// an SM reads (8 against 16 warps, us per call: FP8, 113 KB a projection and SM
// 17.1, 17.7; NVFP4, 225 KB 42.5, 32.9), and what fits beside long rows: 8
// rows of an operand in one part, 6 (FP8) or 8 (NVFP4) in two (20 tokens top-4
// on 16 experts 1024 x 4096, the down-projection with 8 and 16 warps: FP8 48.9,
// 41.6; NVFP4 44.3, 39.9).
// Calls go(GMAX, W).
template <int FMT, int MODE, typename F>
auto by_size(const DeviceInfo& di, const Args& a, int columns, int64_t weight_bytes, F&& go) {
    using std::integral_constant;
    const bool small = weight_bytes < di.num_sms * 160ll * 1024;
    const bool long_rows = PARTS<MODE> * operand_pitch<FMT>(a.w.K) * 8 > (PARTS<MODE> == 2 ? 140 : 112) * 1024;
    if ((columns <= 8 && small) || long_rows) return go(integral_constant<int, 1>(), integral_constant<int, 8>());
    if (columns <= 8) return go(integral_constant<int, 1>(), integral_constant<int, 16>());
    return go(integral_constant<int, 2>(), integral_constant<int, 16>());
}
template <int FMT, int MODE>
int launch_few_by_size(const DeviceInfo& di, const Args& a, int columns, int64_t weight_bytes, cudaStream_t st) {
    return by_size<FMT, MODE>(di, a, columns, weight_bytes,
                              [&](auto g, auto w) { return launch_few<FMT, MODE, decltype(g)::value, decltype(w)::value>(di, a, st); });
}

// DENSE: tokens of a job (with fewer than all, every job streams and widens all weights); 0: none can be staged.
inline int job_tokens(const DeviceInfo& di, Args a, int64_t weight_bytes) {
    return by_size<NVFP4, DENSE>(di, a, a.S, weight_bytes, [&](auto g, auto w) {
        constexpr int columns = 8 * decltype(g)::value;
        if (!stage_plan<NVFP4, DENSE, decltype(g)::value, decltype(w)::value>(di, a)) return 0;
        const int most = a.P < columns ? a.P : columns;
        return a.S < most ? a.S : most;
    });
}

template <int FMT>
int run_moe(const DeviceInfo& di, const __nv_bfloat16* x, const int32_t* ids, const float* tw, int T, int topk, int E,
            const Weights& up, const Weights& down, __nv_bfloat16* y, uint8_t* ws, cudaStream_t st) {
    Args a{};
    int rc = device_status_word(&a.status);
    if (rc) return rc;
    const int S = T * topk;
    float* h = reinterpret_cast<float*>(ws);
    float* o = reinterpret_cast<float*>(ws + align256(4ll * S * up.N));
    a.in = x;
    a.w = up;
    a.ids = ids;
    a.tw = tw;
    a.E = E;
    a.S = S;
    a.T = T;
    a.topk = topk;
    a.out = h;
    // one pass for 16 slots of an expert when their mean calls for it (us a call
    // on 64 experts, top-8, 2048 x 1024; 8 against 16 slots in both projections,
    // h in one part): FP8 mean 4: 57.0, 61.8; 8: 65.6, 74.3; 16: 102, 88.8; NVFP4
    // mean 4: 46.8, 49.2; 8: 64.3, 60.6. The down-projection with h in two parts
    // (8, 16): FP8 mean 12: 81.0, 83.7; 16: 98.0, 101.6, but 24.0, 20.8 on 16
    // experts 1024 x 512; NVFP4 mean 8: 60.6, 64.5; 12: 77.3, 77.5; 16 on 16
    // experts 24.2, 21.6; 32: 46.9, 37.5.
    const int columns = S <= (FMT == FP8 ? 10 : 6) * E ? 8 : 16;
    const int64_t weight_bytes = static_cast<int64_t>(S < E ? S : E) * up.N * up.K / (FMT == FP8 ? 1 : 2);
    if ((rc = launch_few_by_size<FMT, UP>(di, a, columns, weight_bytes, st))) return rc;
    a.in = h;
    a.w = down;
    // few slots: every CTA stages all of h and owns rows of the output, which
    // saves a launch. Against DOWN, us a call in a graph (FP8): 8 slots 2048 x 1024
    // 12.6, 14.2, 512 x 256 7.7, 8.5; 16 slots 2048 x 1024 19.3, 20.1, 2048 x 512
    // 13.3, 14.2, but 1024 x 512 11.2, 10.3 and 15 slots 1040 x 528 13.5, 11.7,
    // which calls from the host turn round (12.7, 15.0 and 14.0, 15.1); 24 slots
    // 1024 x 512 14.2, 12.2, 48 slots 512 x 256 17.2, 11.2.
    if (S <= 16 && PARTS<OWN> * S * operand_pitch<FMT>(down.K) <= 80 * 1024) {
        a.out = y;
        return launch_few<FMT, OWN, 1, 8>(di, a, st);
    }
    a.out = o;
    if ((rc = launch_few_by_size<FMT, DOWN>(di, a, S <= 10 * E ? 8 : 16, weight_bytes, st))) return rc;
    return cuda_check(launch_pdl(combine_kernel, dim3((down.N + 511) / 512, T), dim3(128), 0, st, 1,
                                 static_cast<const float*>(o), ids, tw, topk, E, down.N, y),
                      "few-token combine launch");
}

}  // namespace few

// metis_nvfp4_w4a16_gemm by its tokens, measured on B200 (us; N x K):
//                        6144x2048   14336x4096   2048x6144   1024x1024   4096x14336
//     1  streamed             5.2        10.5         4.9         3.7        12.2
//        tensor cores         8.2        20.8         8.2         4.1        20.0
//     8  streamed             6.8        13.7         9.6         4.4        30.9
//        tensor cores         8.2        20.7         8.3         4.3        20.0
//    16  streamed             8.3        18.9        13.3         4.9        55.5
//        tensor cores         8.3        20.8         8.5         4.4        20.2
//    32  streamed            21.6        52.5
//        tensor cores         8.5        21.0
//  2048  tensor cores        44.0       178          39.2         9.3
//        widened first       50.1       199          51.7        13.3
//  3000  tensor cores        61.1                    67 - 72     12.3
//        widened first       63.0                    79 - 85     14.8
//  4096  tensor cores        90.9                    80          14.2
//        widened first       82.5                    84          17.8
// The border by tokens alone is right for the wide matrix; the two small ones
// would still be 5 and 20% faster without the widening at 4096 tokens.
constexpr int64_t kStreamTokens = 16, kWidenTokens = 3000;

// Up to kStreamTokens, by estimates fitted to the table, in ns: 3000 + 100 per
// 1024 operand values that a CTA stages (a job's) + the codes at 3.2 TB/s, once
// for every job (long rows: fewer tokens fit shared memory) + 500 for a second
// group of columns, against 3750 + 530 per stage. Two jobs, us, streamed and
// tensor cores: 16 x 14336 x 4352 26.9, 22.0; 13 x 12288 x 5632 31.7, 27.3; 9 x
// 14336 x 7104 37.8, 35.6; 16 x 9600 x 5120 25.1, 24.9; 16 x 9600 x 8192 31.2,
// 37.5; 9 x 9600 x 8192 32.2, 37.5; 6 x 9600 x 13632 50.5, 63.6.
static bool nvfp4_w4a16_streams(const DeviceInfo& di, const few::Args& a, const W4a16Plan& plan) {
    const int64_t M = a.S, N = a.w.N, K = a.w.K;
    if (M > kStreamTokens) return false;
    const int64_t job = few::job_tokens(di, a, N * K / 2);
    return job > 0 && job * K * 100 / 1024 + (M + job - 1) / job * (N * K / 6400) + (job > 8 ? 500 : 0) < 750 + 530 * plan.stages;
}

size_t nvfp4_w4a16_workspace(int64_t M, int64_t N, int64_t K) {
    return M <= kWidenTokens ? 0 : static_cast<size_t>(few::align256(2 * N * K) + few::align256(4 * N));
}

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
    return few::run_moe<few::FP8>(di, static_cast<const __nv_bfloat16*>(x_bf16), topk_ids, topk_w, static_cast<int>(T),
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
    return few::run_moe<few::NVFP4>(di, static_cast<const __nv_bfloat16*>(x_bf16), topk_ids, topk_w, static_cast<int>(T),
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    few::Args a{};
    a.in = x_bf16;
    a.w = few::Weights{qb, sfb, gb, static_cast<int>(N), static_cast<int>(K)};
    a.E = 1;
    a.S = a.T = static_cast<int>(M);
    a.topk = 1;
    a.out = y_bf16;
    if (M <= kWidenTokens) {
        W4a16Plan plan;
        if ((rc = plan_nvfp4_w4a16_tensor(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), &plan))) return rc;
        if (!nvfp4_w4a16_streams(di, a, plan))
            return launch_nvfp4_w4a16_tensor(plan, static_cast<const __nv_bfloat16*>(x_bf16), qb, sfb, gb,
                                             static_cast<__nv_bfloat16*>(y_bf16), static_cast<int>(M), static_cast<int>(N),
                                             static_cast<int>(K), st);
    }
    if (M > kWidenTokens) {
        // many tokens: widen the weights once, then the BF16 CTA-pair GEMM
        __nv_bfloat16* wide = static_cast<__nv_bfloat16*>(workspace);
        float* col = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + few::align256(2 * N * K));
        const int64_t blocks = N * K / 16;
        if (blocks > 0xFFFFFFFFll)
            return fail(METIS_ERR_UNSUPPORTED, "nvfp4_w4a16_gemm: N * K too large (N=%lld K=%lld)", (long long)N, (long long)K);
        int64_t grid = (blocks + 256 * few::WIDEN_BATCH - 1) / (256 * few::WIDEN_BATCH);
        if (grid > 8ll * di.num_sms) grid = 8ll * di.num_sms;
        rc = cuda_check(launch_pdl(few::widen_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, 1, qb, sfb, gb,
                                   static_cast<uint32_t>(blocks), static_cast<uint32_t>(K / 16),
                                   0xFFFFFFFFu / static_cast<uint32_t>(K / 16), static_cast<int>(N),
                                   reinterpret_cast<uint4*>(wide), col),
                        "nvfp4 widening launch");
        if (rc) return rc;
        return launch_bf16_gemm(static_cast<const __nv_bfloat16*>(x_bf16), wide, static_cast<__nv_bfloat16*>(y_bf16),
                                static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), col, st);
    }
    if ((rc = device_status_word(&a.status))) return rc;
    return few::launch_few_by_size<few::NVFP4, few::DENSE>(di, a, a.S, N * K / 2, st);
}
