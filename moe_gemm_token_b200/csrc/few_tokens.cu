// Default maths for few tokens with the weights read once: the routed-expert
// layer with FP8 or NVFP4 experts, and the NVFP4 weight-only product.
//   h[s] = W_up[e] x[t],  o[s] = W_down[e] h[s],  y[t] = bf16( sum_j w[t, j] o[t, j] )
// for the slots s = (t, j) with expert e = topk_ids[t, j]; FP32 sums, h and o
// kept in FP32.
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

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int DEPTH = 6;         // pieces in flight per warp

enum Mode { UP = 0, DOWN = 1, OWN = 2, DENSE = 3 };

// Per-format geometry. A piece is 16 rows by 64 bytes: lane (g, t) = (lane / 4,
// lane % 4) holds bytes 16 t .. 16 t + 15 of rows g and g + 8.
template <int FMT>
struct Geo {
    static constexpr int EL = FMT == FP8 ? 64 : 128;     // elements of K per piece
    static constexpr int CH = EL / 32;                   // 8-element chunks of K per lane
    static constexpr int SLOT = 1024 + (FMT == FP8 ? 0 : 256);  // bytes of a piece in the ring
};

struct Args {
    const void* in;        // UP, DENSE: BF16 [tokens, K]; DOWN, OWN: FP32 [S, K]
    Weights w;
    const int32_t* ids;    // [S]; DENSE: null
    const float* tw;       // OWN: [S] routing weights
    int E, S, T, topk;     // DENSE: E = 1, S = T = tokens
    int P;                 // rows of the operand staged at a time
    int pitch;             // bytes between staged rows: 64 mod 128
    void* out;             // UP, DOWN: FP32 [S, N]; OWN: BF16 [T, N]; DENSE: BF16 [T, N]
    uint32_t* status;
};

// Shared memory: ring | partial sums | staged operand | its scales | routing.
struct Smem {
    int part, x, unshift, route, own, total;
};
__host__ __device__ inline Smem smem_layout(int slot_bytes, int gmax, int P, int pitch, int E, int S, bool routed,
                                            bool own) {
    Smem s;
    s.part = WARPS * DEPTH * slot_bytes;
    s.x = s.part + 2 * WARPS * 512 * gmax;
    s.unshift = s.x + P * pitch;
    s.route = s.unshift + ((P * 4 + 15) & ~15);
    s.own = s.route + (routed ? 4 * (E + 2 * (E < S ? E : S) + 2 + S) + 16 : 16);
    s.own = (s.own + 15) & ~15;
    s.total = s.own + (own ? S * 16 * 4 : 0);
    return s;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
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

// Eight elements of an operand row as FP32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// One warp stages one operand row [K] as FP16 after the power-of-two shift
// that brings its largest magnitude into [2^14, 2^15) (exact for BF16 values
// within 2^-29 of the largest; FP32 values are rounded to 11 significant
// bits). A row with an infinity or a NaN is not shifted. 16-byte chunks are
// stored in the order in which the lanes read them (operand_chunk), zeros
// from K to the end of the last piece.
template <int FMT>
__device__ __forceinline__ int operand_chunk(int q) {
    constexpr int C = Geo<FMT>::CH;  // the piece's chunk t * C + i is stored at i * 4 + t
    const int piece = q / (4 * C), r = q % (4 * C);
    return piece * 4 * C + (r % C) * 4 + r / C;
}
template <int FMT, typename In>
__device__ __forceinline__ void stage_row(const In* row, int K, uint8_t* dst, float* unshift, int lane) {
    const int chunks = K / 8;
    uint32_t m = 0;
    for (int q = lane; q < chunks; q += 32) {
        float v[8];
        load8(row + 8 * q, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const int sh = m == 0 || m >= 0x7F800000u ? 0 : 14 - ilogbf(__uint_as_float(m));
    // 2^sh may leave FP32's range: two factors
    const int sa = max(-100, min(100, sh));
    const float fa = pow2(sa), fb = pow2(sh - sa);
    if (lane == 0) *unshift = ldexpf(1.0f, -sh);
    constexpr int PC = Geo<FMT>::EL / 8;
    const int padded = (chunks + PC - 1) / PC * PC;
    for (int q = lane; q < padded; q += 32) {
        uint4 o = make_uint4(0, 0, 0, 0);
        if (q < chunks) {
            float v[8];
            load8(row + 8 * q, v);
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 p = __floats2half2_rn(v[2 * i] * fa * fb, v[2 * i + 1] * fa * fb);
                h[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
            o = make_uint4(h[0], h[1], h[2], h[3]);
        }
        *reinterpret_cast<uint4*>(dst + 16 * operand_chunk<FMT>(q)) = o;
    }
}

// The chosen experts in ascending order, and the slots of each.
struct Routing {
    int* expert;   // [active]
    int* start;    // [active + 1] first entry of each in slots
    int* slots;    // [S]
    int active;
};

// Built by every CTA from the ids: counts, then a scan over the experts. The
// order of an expert's slots does not matter (a slot is a column of the MMA).
__device__ __forceinline__ Routing build_routing(const Args& a, uint8_t* mem) {
    int* count = reinterpret_cast<int*>(mem);                 // [E], then first entries
    const int most = a.E < a.S ? a.E : a.S;
    Routing r;
    r.expert = count + a.E;
    r.start = r.expert + most;
    r.slots = r.start + most + 1;
    int* active = r.slots + a.S;
    for (int e = threadIdx.x; e < a.E; e += THREADS) count[e] = 0;
    __syncthreads();
    int id[MAX_S / THREADS], rank[MAX_S / THREADS];
#pragma unroll
    for (int i = 0; i < MAX_S / THREADS; ++i) {
        const int s = threadIdx.x + i * THREADS;
        id[i] = -1;
        if (s < a.S) {
            const int e = a.ids[s];
            if (e >= 0 && e < a.E) {
                id[i] = e;
                rank[i] = atomicAdd(&count[e], 1);
            } else if (blockIdx.x == 0) {
                atomicOr(a.status, kDevErrBadIndex);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int na = 0, tot = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int c = e0 + lane < a.E ? count[e0 + lane] : 0;
            const unsigned m = __ballot_sync(0xffffffffu, c > 0);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (c > 0) {
                const int at = na + __popc(m & ((1u << lane) - 1u));
                r.expert[at] = e0 + lane;
                r.start[at] = tot + incl - c;
                count[e0 + lane] = tot + incl - c;
            }
            na += __popc(m);
            tot += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            r.start[na] = tot;
            *active = na;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MAX_S / THREADS; ++i)
        if (id[i] >= 0) r.slots[count[id[i]] + rank[i]] = threadIdx.x + i * THREADS;
    r.active = *active;
    __syncthreads();
    return r;
}

template <int FMT, int MODE, int GMAX>
__global__ void __launch_bounds__(THREADS, 2) few_kernel(const Args a) {
    using G = Geo<FMT>;
    using In = typename std::conditional<MODE == UP || MODE == DENSE, __nv_bfloat16, float>::type;
    extern __shared__ __align__(128) uint8_t smem[];
    const Smem L = smem_layout(G::SLOT, GMAX, a.P, a.pitch, a.E, a.S, MODE != DENSE, MODE == OWN);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane >> 2, t = lane & 3;
    const int N = a.w.N, K = a.w.K;
    const int row_bytes = FMT == FP8 ? K : K / 2;
    const int kp = (row_bytes + 63) / 64;  // pieces per tile of rows
    float* part = reinterpret_cast<float*>(smem + L.part);
    uint8_t* xs = smem + L.x;
    float* unshift = reinterpret_cast<float*>(smem + L.unshift);

    // UP, DENSE: the ids or the operand may be the previous kernel's output.
    // DOWN, OWN: only the up-projection can still be running (it lets this
    // grid start after its own wait), so the routing and the weights may be
    // read before the wait, h not.
    if constexpr (MODE == UP || MODE == DENSE) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    Routing rt{};
    if constexpr (MODE == DENSE) rt.active = 1;
    else rt = build_routing(a, smem + L.route);

    // The rows of this CTA: UP, DOWN, DENSE: an even share of the chosen
    // experts' rows one after another; OWN: an even share of the output's
    // rows, for every chosen expert.
    const int64_t total = MODE == OWN ? N : static_cast<int64_t>(rt.active) * N;
    const int64_t r0 = total * blockIdx.x / gridDim.x, r1 = total * (blockIdx.x + 1) / gridDim.x;
    const int first = MODE == OWN ? 0 : static_cast<int>(r0 / N);
    const int own_tiles = static_cast<int>((r1 - r0 + 15) / 16);
    const int nseg = r1 <= r0 ? 0 : MODE == OWN ? own_tiles * rt.active : static_cast<int>((r1 - 1) / N) - first + 1;
    // The warps split K (ks of them share a tile of 16 rows) and, when K is
    // short and there are tiles enough, the tiles (teams).
    int ks = WARPS;
    if (MODE != OWN)
        while (ks > 1 && kp < 4 * ks && own_tiles >= 8 * WARPS / ks) ks >>= 1;
    const int teams = WARPS / ks, team = warp / ks, kslice = warp % ks;

    struct Seg { int e, start, n, pb, pe; };
    auto segment = [&](int s) {
        Seg sg;
        int x = 0;
        if constexpr (MODE == OWN) {
            x = s % rt.active;
            sg.pb = static_cast<int>(r0) + 16 * (s / rt.active);
            sg.pe = min(sg.pb + 16, static_cast<int>(r1));
        } else {
            x = first + s;
            const int64_t b = static_cast<int64_t>(x) * N;
            sg.pb = static_cast<int>(max(r0 - b, static_cast<int64_t>(0)));
            sg.pe = static_cast<int>(min(r1 - b, static_cast<int64_t>(N)));
        }
        if constexpr (MODE == DENSE) {
            sg.e = 0, sg.start = 0, sg.n = a.S;
        } else {
            sg.e = rt.expert[x];
            sg.start = rt.start[x];
            sg.n = rt.start[x + 1] - sg.start;
        }
        return sg;
    };
    const int pass_rows = min(a.P, 8 * GMAX);

    // ---- weight stream: this warp's pieces in order, DEPTH of them in flight
    // in lane-private places of the ring (a lane reads back what it copied)
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * DEPTH * G::SLOT);
    int is = -1, ipass = 0, inpass = 0, itile = 0, intiles = 0, ik = kp;  // the next piece to request
    Seg iseg{};
    const uint8_t* wp[2];
    const uint8_t* sp[2];
    bool wv[2] = {false, false};
    auto request = [&](int slot) {
        if (ik >= kp) {  // next tile of this team
            itile += teams;
            while (itile >= intiles) {
                if (++ipass >= inpass) {
                    if (++is >= nseg) break;
                    iseg = segment(is);
                    ipass = 0;
                    inpass = (iseg.n + pass_rows - 1) / pass_rows;
                    intiles = (iseg.pe - iseg.pb + 15) / 16;
                }
                itile = team;
            }
            ik = kslice;
            if (is < nseg) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = iseg.pb + 16 * itile + 8 * h + g;
                    wv[h] = p < iseg.pe;
                    const int64_t row = static_cast<int64_t>(iseg.e) * N + place_to_row<FMT>(wv[h] ? p : iseg.pb);
                    wp[h] = a.w.q + row * row_bytes + 16 * t;
                    if constexpr (FMT == NVFP4)
                        sp[h] = a.w.sf + ((row >> 7) * (K / 64) + (t >> 1)) * 512 + 16 * (row & 31) + 4 * ((row & 127) >> 5);
                }
            } else {
                ik = kp;
                itile = 0, intiles = 0, ipass = 0, inpass = 0;  // nothing left: stay here
                is = nseg;
            }
        }
        if (is < nseg && ik < kp) {
            const uint32_t dst = ring + slot * G::SLOT + 16 * lane;
            const bool in = 64 * ik + 16 * t < row_bytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool v = wv[h] && in;
                cp_async16(dst + 512 * h, v ? wp[h] + 64 * ik : a.w.q, v);
                if constexpr (FMT == NVFP4)
                    cp_async4(ring + slot * G::SLOT + 1024 + 128 * h + 4 * lane, v ? sp[h] + 1024 * static_cast<int64_t>(ik) : a.w.sf, v);
            }
            ik += ks;
        }
        cp_async_commit();
    };
    for (int d = 0; d < DEPTH; ++d) request(d);
    int slot = 0;

    if constexpr (MODE == DOWN || MODE == OWN) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    // ---- operand rows
    auto stage = [&](int start, int n) {
        for (int i = warp; i < n; i += WARPS) {
            const int s = MODE == DENSE ? start + i : rt.slots[start + i];
            const int64_t r = MODE == UP ? s / a.topk : s;
            stage_row<FMT>(static_cast<const In*>(a.in) + r * K, K, xs + i * a.pitch, unshift + i, lane);
        }
    };
    if constexpr (MODE == OWN) {
        stage(0, rt.active ? rt.start[rt.active] : 0);
        __syncthreads();
    }

    int buf = 0;
    for (int s = 0; s < nseg; ++s) {
        const Seg sg = segment(s);
        const int ntiles = (sg.pe - sg.pb + 15) / 16;
        for (int p0 = 0; p0 < sg.n; p0 += pass_rows) {
            const int n = min(pass_rows, sg.n - p0);
            const int ng = (n + 7) / 8;
            const int xrow0 = MODE == OWN ? sg.start + p0 : 0;
            if constexpr (MODE != OWN) {
                __syncthreads();
                stage(sg.start + p0, n);
                __syncthreads();
            }
            for (int tile0 = 0; tile0 < ntiles; tile0 += teams) {
                float acc[GMAX][4];
#pragma unroll
                for (int q = 0; q < GMAX; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.0f;
                if (tile0 + team < ntiles) {
                    for (int k = kslice; k < kp; k += ks) {
                        cp_async_wait_oldest();
                        const uint8_t* src = smem + warp * DEPTH * G::SLOT + slot * G::SLOT;
                        const uint4 wa = *reinterpret_cast<const uint4*>(src + 16 * lane);
                        const uint4 wb = *reinterpret_cast<const uint4*>(src + 512 + 16 * lane);
                        uint32_t sa = 0, sb = 0;
                        if constexpr (FMT == NVFP4) {
                            sa = *reinterpret_cast<const uint32_t*>(src + 1024 + 4 * lane) >> (16 * (t & 1));
                            sb = *reinterpret_cast<const uint32_t*>(src + 1152 + 4 * lane) >> (16 * (t & 1));
                        }
                        // the piece's weights as the MMAs' A operand: rows g, g + 8; four K elements a step
                        constexpr int STEPS = G::EL / 16;
                        uint32_t A[STEPS][4];
                        if constexpr (FMT == FP8) {
                            const uint32_t va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                e4m3x4_to_f16(va[i], A[i][0], A[i][2]);
                                e4m3x4_to_f16(vb[i], A[i][1], A[i][3]);
                            }
                        } else {
                            const uint32_t va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
                            uint32_t fa[2], fb[2];
                            scale_pairs(sa, fa[0], fa[1]);
                            scale_pairs(sb, fb[0], fb[1]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t ha[4], hb[4];
                                e2m1x8_to_f16(va[i], ha);
                                e2m1x8_to_f16(vb[i], hb);
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    A[2 * i + j][0] = mul_f16x2(ha[2 * j], fa[i / 2]);
                                    A[2 * i + j][2] = mul_f16x2(ha[2 * j + 1], fa[i / 2]);
                                    A[2 * i + j][1] = mul_f16x2(hb[2 * j], fb[i / 2]);
                                    A[2 * i + j][3] = mul_f16x2(hb[2 * j + 1], fb[i / 2]);
                                }
                            }
                        }
                        request(slot);
                        slot = slot + 1 == DEPTH ? 0 : slot + 1;
#pragma unroll
                        for (int q = 0; q < GMAX; ++q) {
                            if (q >= ng) break;
                            const bool have = 8 * q + g < n;
                            const uint8_t* xr = xs + (xrow0 + 8 * q + g) * a.pitch + k * (2 * G::EL) + 16 * t;
#pragma unroll
                            for (int i = 0; i < G::CH; ++i) {
                                uint4 xv = make_uint4(0, 0, 0, 0);
                                if (have) xv = *reinterpret_cast<const uint4*>(xr + 64 * i);
                                mma_16816(acc[q], A[2 * i][0], A[2 * i][1], A[2 * i][2], A[2 * i][3], xv.x, xv.y);
                                mma_16816(acc[q], A[2 * i + 1][0], A[2 * i + 1][1], A[2 * i + 1][2], A[2 * i + 1][3], xv.z, xv.w);
                            }
                        }
                    }
                }
                // ---- the warps' sums meet in shared memory, added in a fixed order
                float* pb = part + buf * (WARPS * 128 * GMAX);
#pragma unroll
                for (int q = 0; q < GMAX; ++q)
                    if (q < ng)
                        *reinterpret_cast<float4*>(pb + (warp * GMAX + q) * 128 + 4 * lane) =
                            make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
                __syncthreads();
                for (int o = threadIdx.x; o < teams * ng * 128; o += THREADS) {
                    const int tm = o / (ng * 128), q = (o >> 7) % ng, at = o & 127;
                    const int ln = at >> 2, comp = at & 3;
                    const int col = 8 * q + 2 * (ln & 3) + (comp & 1);
                    const int p = sg.pb + 16 * (tile0 + tm) + (ln >> 2) + 8 * (comp >> 1);
                    if (col >= n || p >= sg.pe) continue;
                    float sum = 0.0f;
                    for (int w = 0; w < ks; ++w) sum += pb[((tm * ks + w) * GMAX + q) * 128 + at];
                    const int row = place_to_row<FMT>(p);
                    const float sc = FMT == FP8 ? a.w.s[static_cast<int64_t>(sg.e) * N + row] : a.w.s[sg.e];
                    const float v = sum * unshift[xrow0 + col] * sc;
                    if constexpr (MODE == DENSE) {
                        static_cast<__nv_bfloat16*>(a.out)[static_cast<int64_t>(p0 + col) * N + row] = __float2bfloat16_rn(v);
                    } else {
                        const int sl = rt.slots[sg.start + p0 + col];
                        if constexpr (MODE == OWN) reinterpret_cast<float*>(smem + L.own)[sl * 16 + (p - sg.pb)] = v;
                        else static_cast<float*>(a.out)[static_cast<int64_t>(sl) * N + row] = v;
                    }
                }
                buf ^= 1;
            }
        }
        if constexpr (MODE == OWN) {
            if (s % rt.active == rt.active - 1) {
                // every chosen expert has given its part of these rows
                __syncthreads();
                const float* ov = reinterpret_cast<const float*>(smem + L.own);
                for (int i = threadIdx.x; i < a.T * 16; i += THREADS) {
                    const int tk = i >> 4, p = sg.pb + (i & 15);
                    if (p >= sg.pe) continue;
                    float y = 0.0f;
                    for (int j = 0; j < a.topk; ++j) {
                        const int sl = tk * a.topk + j;
                        const int e = a.ids[sl];
                        if (e >= 0 && e < a.E) y = fmaf(a.tw[sl], ov[sl * 16 + (i & 15)], y);
                    }
                    static_cast<__nv_bfloat16*>(a.out)[static_cast<int64_t>(tk) * N + place_to_row<FMT>(p)] = __float2bfloat16_rn(y);
                }
                __syncthreads();
            }
        }
    }
    if constexpr (MODE == OWN) {
        if (rt.active == 0) {  // no token has an expert
            for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < static_cast<int64_t>(a.T) * N;
                 i += static_cast<int64_t>(gridDim.x) * THREADS)
                static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(0.0f);
        }
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

// Launches few_kernel with as much of the operand staged as fits: two CTAs per
// SM when at least `want` rows (or 8) fit beside the ring, else one.
template <int FMT, int MODE, int GMAX>
int launch_few(const DeviceInfo& di, Args a, int want, cudaStream_t st) {
    using G = Geo<FMT>;
    static std::atomic<uint64_t> done[64];
    int rc = once_per_context(done, di.device, [&] {
        return cuda_check(cudaFuncSetAttribute(few_kernel<FMT, MODE, GMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               di.max_smem_optin),
                          "cudaFuncSetAttribute(few tokens)");
    });
    if (rc) return rc;
    a.pitch = (a.w.K + G::EL - 1) / G::EL * G::EL * 2 + 64;
    constexpr int HALF = 112 * 1024;  // two CTAs per SM
    auto bytes = [&](int P) { return smem_layout(G::SLOT, GMAX, P, a.pitch, a.E, a.S, MODE != DENSE, MODE == OWN).total; };
    const int base = bytes(0) + 16;
    int P = (HALF - base) / (a.pitch + 4), per_sm = 2;
    if (P < want && P < 8) {
        P = (di.max_smem_optin - base) / (a.pitch + 4);
        per_sm = 1;
    }
    if (P < 1 || (MODE == OWN && P < want)) return fail(METIS_ERR_UNSUPPORTED, "few-token kernel: K=%d too long", a.w.K);
    a.P = P < want ? P : want;
    return cuda_check(launch_pdl(few_kernel<FMT, MODE, GMAX>, dim3(di.num_sms * per_sm), dim3(THREADS), bytes(a.P), st, 1, a),
                      "few-token kernel launch");
}

// By the tokens that one pass multiplies (8, 16 or 32).
template <int FMT, int MODE>
int launch_few_by_rows(const DeviceInfo& di, const Args& a, int rows, int want, cudaStream_t st) {
    if (rows <= 8) return launch_few<FMT, MODE, 1>(di, a, want, st);
    if (rows <= 16) return launch_few<FMT, MODE, 2>(di, a, want, st);
    return launch_few<FMT, MODE, 4>(di, a, want, st);
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
    const int rows = S < T ? S : T;  // of one expert, unless a token names it twice
    const int most = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    if ((rc = launch_few_by_rows<FMT, UP>(di, a, rows, S < most ? S : most, st))) return rc;
    a.in = h;
    a.w = down;
    // few slots: every CTA stages all of h and owns rows of the output
    const int pitch = (down.K + Geo<FMT>::EL - 1) / Geo<FMT>::EL * Geo<FMT>::EL * 2 + 64;
    if (S <= 64 && S * pitch <= 40 * 1024) {
        a.out = y;
        return launch_few<FMT, OWN, 1>(di, a, S, st);
    }
    a.out = o;
    if ((rc = launch_few_by_rows<FMT, DOWN>(di, a, rows, S < most ? S : most, st))) return rc;
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
    few::Args a{};
    if ((rc = device_status_word(&a.status))) return rc;
    a.in = x_bf16;
    a.w = few::Weights{qb, sfb, gb, static_cast<int>(N), static_cast<int>(K)};
    a.E = 1;
    a.S = a.T = static_cast<int>(M);
    a.topk = 1;
    a.out = y_bf16;
    const int rows = static_cast<int>(M < 32 ? M : 32);
    return few::launch_few_by_rows<few::NVFP4, few::DENSE>(di, a, rows, rows, static_cast<cudaStream_t>(stream));
}
