// Decode attention over the paged cache: dense, with a shared prefix, or over
// listed pages.
//
// Mathematics.  For each query, o = sum_t p_t v_t / sum_t p_t with
// p_t = 2^(s_t - m), s_t the scaled score in log2 units and m a reference that
// only moves when a score passes it by 8 (one pass over the rows).  Rows come in
// cells of 16 rows of one KV head; a warp takes a cell at a time and multiplies
// it on the tensor cores (mma.m16n8k16): S = Q K^T with query rows as M, then
// O^T += V^T P^T with 16 elements as M and 8 queries as N.  The cell layout is
// the operands' register layout, so a lane's loads are its fragments, K and V
// codes turn into fp16 pairs in registers, and S's accumulators are P^T's B
// fragments as they stand: nothing is transposed or passed through shared
// memory on the way.
//   K: codes are small integers, exact in fp16, so the products with the query
//      run on codes and each 32-element block's sum is scaled by its d in f32.
//   V: v = u d + m in one half2 fma a pair of rows (one rounding to fp16).
// Tiles of 8 or 16 queries of bf16 (the tile is taken by the most queries that
// a key has); f32 queries keep f32 accuracy: rows 0..7 of an S tile
// carry the high part of the queries and rows 8..15 the low part, two fp16
// numbers (22 bits of a query scaled to its largest element), and P d goes in as
// three bf16 numbers (all its 24 bits; two left outputs off by up to 3e-6 of their
// size where f32 arithmetic leaves 1e-6) against the exact codes u - 16, with
// sum p (m + 16 d) kept in f32 beside it.
//
// Why tensor cores for one token: the products cost the same for 1 or 8 queries,
// so the work that grows with the bytes is the unpacking alone, where the
// multiply-add form needs as many instructions again for each 4 queries.
//
// Work is cut stream-K fashion: see kvq_paged.cuh.
//
// Measured (q8_0 / q5_1, bf16, 32 query and 8 KV heads of 128): 64 sequences of 1024
// to 16384 rows 191 us, 0.80 of the copy rate, bound by some 520 instructions a
// cell; one of 32768 rows 23 us and one of 512 (8 query and 2 KV heads) 12 us, of
// which 11 are the start and the end: plan, first lookups and copies, joins,
// records, and fetching code that runs once.
#include "kvq_device.cuh"
#include "kvq_paged.cuh"
#include "kvq_paged_work.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

namespace kvq {
namespace paged {
namespace {


// Query tiles: 8 or 16 bf16 queries, or 8 or 16 of f32 in two parts
enum Tile { kT8 = 0, kT16 = 1, kF32 = 2, kF32W = 3 };
template <int TILE>
constexpr bool two_parts() { return TILE == kF32 || TILE == kF32W; }

// Warps of a CTA (one CTA an SM): as many as the accumulators leave registers for
template <int NB, int TILE>
constexpr int warps_of() { return NB == 8 ? 8 : NB == 4 && (TILE == kT16 || TILE == kF32W) ? 12 : 16; }
// Groups of four warps, which work on ranges of their own where there is enough work
template <int NB, int TILE>
constexpr int groups_of() { return warps_of<NB, TILE>() / 4; }
template <int TILE>
constexpr int queries_of() { return TILE == kT16 || TILE == kF32W ? 16 : 8; }

// c = a b + z (z: four zeros that stay in registers, where a constant would be
// written to four new ones for each product)
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1, const float (&z)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// code bytes (biased by 128) sel of w under the exponent of 1024, minus 1152: exact
__device__ __forceinline__ uint32_t k_pair(uint32_t w, uint32_t sel, uint32_t exps) {
    return as_u32(__hsub2(as_h2(__byte_perm(w, exps, sel)), as_h2(0x64806480u)));
}
__device__ __forceinline__ float load_q(const void* q, long long idx, int bf16) {
    if (bf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[idx]);
    return reinterpret_cast<const float*>(q)[idx];
}

// ------------------------------------------------------------ split kernel

template <int NB, bool F8, int TILE>
struct Acc {
    static constexpr int NQ = queries_of<TILE>() / 8;     // groups of 8 queries
    // O^T tile 2b + rp of a group: rows g / g + 8 are elements 32b + 4g + 2rp and
    // + 1, columns 2j, 2j + 1 queries: [0] (el, 2j) [1] (el, 2j+1) [2] (el+1, 2j) ..
    float o[NQ][2 * NB][4];
    float m[NQ], l[NQ];                                   // query g (+ 8): reference, sum of p
    float mt[NQ][two_parts<TILE>() && !F8 ? NB : 1];      // sum p (m + 16 d) of query g (+ 8)
};

// The queries of a fragment: factor of a score, rows seen
struct RowInfo {
    float fac[16];
    int lo[16], hi[16];
    int bad[16];                                          // not finite
};

// What a lane keeps of them: queries g (+ 8), and the extremes over all
template <int NQ>
struct LaneRows {
    float fac[NQ];
    int lo[NQ], hi[NQ];
    int lo_min, lo_max, hi_min, hi_max;
};

// Values of rows that no query sees, in the staged cell: zeroed, for they may be any bytes
template <int NB, bool F8, typename Rows>
__device__ __forceinline__ void clear_rows(uint8_t* cell, int row0, const Rows& ri, int lane) {
    if constexpr (F8) {
        const int j = lane & 3;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            uint32_t* p = reinterpret_cast<uint32_t*>(cell + 512 * NB + c * 512 + lane * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = (2 * c + (i >> 1)) / NB;
                const int at = row0 + 8 * h + 2 * j;
                const uint32_t k = (at >= ri.lo_min && at < ri.hi_max ? 0x00ff00ffu : 0u) |
                                   (at + 1 >= ri.lo_min && at + 1 < ri.hi_max ? 0xff00ff00u : 0u);
                p[i] &= k;
            }
        }
    } else {
        for (int i = lane; i < 16 * NB; i += 32) {
            const int t = i & 15, b = i >> 4;
            if (row0 + t >= ri.lo_min && row0 + t < ri.hi_max) continue;
            uint16_t* p = reinterpret_cast<uint16_t*>(cell + 864 * NB + (((t & 7) >> 1) * NB + b) * 16 + (2 * (t >> 3) + (t & 1)) * 2);
            p[0] = 0;
            p[4] = 0;
        }
    }
    __syncwarp();
}

// One staged cell, 16 rows from logical row row0 on, into the warp's accumulators
template <int NB, bool F8, int TILE>
__device__ __forceinline__ void take_cell(const SplitArgs& a, uint8_t* cell, int row0, const uint8_t* __restrict__ qs,
                                          const LaneRows<Acc<NB, F8, TILE>::NQ>& lr, int lane, const float (&zero)[4],
                                          uint32_t magic, uint32_t exps, Acc<NB, F8, TILE>& acc) {
    constexpr bool HL = two_parts<TILE>();
    constexpr int NQ = Acc<NB, F8, TILE>::NQ;
    const int j = lane & 3;
    const bool edge = row0 < lr.lo_max || row0 + 16 > lr.hi_min;
    if (edge) clear_rows<NB, F8>(cell, row0, lr, lane);
    // ---- scores
    float sc[2][2 * NQ];                                  // [rows 2j + 8t + i][2 r + i], query g + 8 r
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2 * NQ; ++i) sc[t][i] = 0.f;
    // query fragments: 16 queries, or (two parts) 8 high parts over their 8 low ones
    constexpr int QF = HL ? NQ : 1;
    float raw[QF][2][4];                                  // E4M3: the products themselves
#pragma unroll
    for (int r = 0; r < QF; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[r][t][i] = 0.f;
    auto q_frag = [&](int r, int step) {
        return *reinterpret_cast<const uint4*>(qs + ((r * 2 * NB + step) * 32 + lane) * 16);
    };
#pragma unroll
    for (int bp = 0; bp < NB / 2; ++bp) {
        uint4 kk[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) kk[t] = *reinterpret_cast<const uint4*>(cell + bp * 1024 + t * 512 + lane * 16);
        uint4 ks;                                         // d of rows (2j, 2j+1), (2j+8, 2j+9), blocks 2bp and 2bp + 1
        if constexpr (!F8) ks = *reinterpret_cast<const uint4*>(cell + 512 * NB + (j * NB + 2 * bp) * 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int b = 2 * bp + e;
            uint4 a0[QF], a1[QF];
#pragma unroll
            for (int r = 0; r < QF; ++r) {
                a0[r] = q_frag(r, 2 * b);
                a1[r] = q_frag(r, 2 * b + 1);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t w0 = e ? kk[t].z : kk[t].x, w1 = e ? kk[t].w : kk[t].y;
                if constexpr (F8) {
                    const uint32_t k0 = f8_pair(w0), k1 = f8_pair(w0 >> 16), k2 = f8_pair(w1), k3 = f8_pair(w1 >> 16);
#pragma unroll
                    for (int r = 0; r < QF; ++r) {
                        mma_f16(raw[r][t], a0[r], k0, k1);
                        mma_f16(raw[r][t], a1[r], k2, k3);
                    }
                } else {
                    const uint32_t k0 = k_pair(w0, 0x4140u, exps), k1 = k_pair(w0, 0x4342u, exps);
                    const uint32_t k2 = k_pair(w1, 0x4140u, exps), k3 = k_pair(w1, 0x4342u, exps);
                    const float2 d = __half22float2(as_h2(e ? (t ? ks.w : ks.z) : (t ? ks.y : ks.x)));
#pragma unroll
                    for (int r = 0; r < QF; ++r) {
                        float c[4];
                        mma_f16_new(c, a0[r], k0, k1, zero);
                        mma_f16(c, a1[r], k2, k3);
                        if constexpr (HL) {
                            c[0] += c[2];
                            c[1] += c[3];
                        }
                        sc[t][2 * r] = fmaf(c[0], d.x, sc[t][2 * r]);
                        sc[t][2 * r + 1] = fmaf(c[1], d.y, sc[t][2 * r + 1]);
                        if constexpr (TILE == kT16) {
                            sc[t][2] = fmaf(c[2], d.x, sc[t][2]);
                            sc[t][3] = fmaf(c[3], d.y, sc[t][3]);
                        }
                    }
                }
            }
        }
    }
    if constexpr (F8) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2 * NQ; ++i) sc[t][i] = HL ? raw[i / 2 % QF][t][i & 1] + raw[i / 2 % QF][t][2 + (i & 1)] : raw[0][t][i];
    }
    // ---- scale, cap, mask; the reference
    float top[NQ];
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) sc[t][2 * r + i] *= lr.fac[r];
        if (a.softcap_b > 0.f) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[t][2 * r + i] = a.softcap_b * tanhf(a.softcap_a * sc[t][2 * r + i]);
        }
        if (edge) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = row0 + 8 * t + 2 * j + i;
                    if (at < lr.lo[r] || at >= lr.hi[r]) sc[t][2 * r + i] = kNegInf;
                }
        }
        top[r] = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
    }
    bool move = top[0] > acc.m[0] + kLazy;
    if (NQ == 2) move |= top[NQ - 1] > acc.m[NQ - 1] + kLazy;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            float v = top[r];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            float al = 1.f;
            if (v > acc.m[r] + kLazy) {
                al = ex2(acc.m[r] - v);
                acc.m[r] = v;
                acc.l[r] *= al;
            }
            if constexpr (HL && !F8) {
#pragma unroll
                for (int b = 0; b < NB; ++b) acc.mt[r][b] *= al;
            }
            const float al0 = __shfl_sync(0xffffffffu, al, 8 * j), al1 = __shfl_sync(0xffffffffu, al, 8 * j + 4);
#pragma unroll
            for (int n = 0; n < 2 * NB; ++n) {
                acc.o[r][n][0] *= al0;
                acc.o[r][n][1] *= al1;
                acc.o[r][n][2] *= al0;
                acc.o[r][n][3] *= al1;
            }
        }
    }
    // ---- probabilities
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
        const float c = kShift - acc.m[r];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) sc[t][2 * r + i] = ex2(sc[t][2 * r + i] + c);
        acc.l[r] += (sc[0][2 * r] + sc[0][2 * r + 1]) + (sc[1][2 * r] + sc[1][2 * r + 1]);
    }
    // ---- values
    uint32_t pb[NQ][2];                                   // B fragments: rows (2j, 2j+1), (2j+8, 2j+9) of query g (+ 8)
    uint32_t pl[NQ][2];                                   // low parts (E4M3 rows, f32 queries)
#pragma unroll
    for (int r = 0; r < NQ; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t) pb[r][t] = as_u32(__floats2half2_rn(sc[t][2 * r], sc[t][2 * r + 1]));
    if constexpr (HL && F8) {
#pragma unroll
        for (int r = 0; r < NQ; ++r)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float2 f = __half22float2(as_h2(pb[r][t]));
                pl[r][t] = as_u32(__floats2half2_rn(sc[t][2 * r] - f.x, sc[t][2 * r + 1] - f.y));
            }
    }
    if constexpr (F8) {
        uint4 vv[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) vv[c] = *reinterpret_cast<const uint4*>(cell + 512 * NB + c * 512 + lane * 16);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int n0 = b, n1 = NB + b;
#pragma unroll
            for (int rp = 0; rp < 2; ++rp) {
                const uint32_t x = n0 & 1 ? (rp ? vv[n0 / 2].w : vv[n0 / 2].z) : (rp ? vv[n0 / 2].y : vv[n0 / 2].x);
                const uint32_t y = n1 & 1 ? (rp ? vv[n1 / 2].w : vv[n1 / 2].z) : (rp ? vv[n1 / 2].y : vv[n1 / 2].x);
                const uint4 va = make_uint4(f8_pair(x), f8_pair(x >> 16), f8_pair(y), f8_pair(y >> 16));
#pragma unroll
                for (int r = 0; r < NQ; ++r) mma_f16(acc.o[r][2 * b + rp], va, pb[r][0], pb[r][1]);
                if constexpr (HL)
#pragma unroll
                    for (int r = 0; r < NQ; ++r) mma_f16(acc.o[r][2 * b + rp], va, pl[r][0], pl[r][1]);
            }
        }
    } else {
        uint32_t u[2 * NB], nb[NB / 2];
#pragma unroll
        for (int c = 0; c < NB / 2; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(cell + 544 * NB + c * 512 + lane * 16);
            u[4 * c] = w.x; u[4 * c + 1] = w.y; u[4 * c + 2] = w.z; u[4 * c + 3] = w.w;
            nb[c] = *reinterpret_cast<const uint32_t*>(cell + 800 * NB + c * 128 + lane * 4);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 dm = *reinterpret_cast<const uint4*>(cell + 864 * NB + (j * NB + b) * 16);
            const int n0 = b, n1 = NB + b;
            if constexpr (!HL) {
                auto value = [&](auto R, int n, uint32_t d, uint32_t m) {
                    constexpr int r = decltype(R)::value;
                    const __half2 c = __hsub2(as_h2(v_codes<r>(u[n], nb[n / 4], n % 4, magic)), as_h2(magic));
                    return as_u32(__hfma2(c, as_h2(d), as_h2(m)));
                };
                const std::integral_constant<int, 0> r0{};
                const std::integral_constant<int, 1> r1{};
                const std::integral_constant<int, 2> r2{};
                const std::integral_constant<int, 3> r3{};
                const uint4 v0 = make_uint4(value(r0, n0, dm.x, dm.z), value(r1, n0, dm.x, dm.z), value(r0, n1, dm.y, dm.w), value(r1, n1, dm.y, dm.w));
#pragma unroll
                for (int r = 0; r < NQ; ++r) mma_f16(acc.o[r][2 * b], v0, pb[r][0], pb[r][1]);
                const uint4 v1 = make_uint4(value(r2, n0, dm.x, dm.z), value(r3, n0, dm.x, dm.z), value(r2, n1, dm.y, dm.w), value(r3, n1, dm.y, dm.w));
#pragma unroll
                for (int r = 0; r < NQ; ++r) mma_f16(acc.o[r][2 * b + 1], v1, pb[r][0], pb[r][1]);
            } else {
                const float2 d0 = __half22float2(as_h2(dm.x)), d1 = __half22float2(as_h2(dm.y));
                const float2 m0 = __half22float2(as_h2(dm.z)), m1 = __half22float2(as_h2(dm.w));
                uint32_t px[3][NQ][2];                     // p d in three bf16 parts, largest first
#pragma unroll
                for (int r = 0; r < NQ; ++r) {
                    const float p0 = sc[0][2 * r], p1 = sc[0][2 * r + 1], p2 = sc[1][2 * r], p3 = sc[1][2 * r + 1];
                    float x0 = p0 * d0.x, x1 = p1 * d0.y, x2 = p2 * d1.x, x3 = p3 * d1.y;
                    float t = acc.mt[r][b];
                    t = fmaf(p0, fmaf(16.f, d0.x, m0.x), t);
                    t = fmaf(p1, fmaf(16.f, d0.y, m0.y), t);
                    t = fmaf(p2, fmaf(16.f, d1.x, m1.x), t);
                    acc.mt[r][b] = fmaf(p3, fmaf(16.f, d1.y, m1.y), t);
                    const __nv_bfloat162 h0 = __floats2bfloat162_rn(x0, x1), h1 = __floats2bfloat162_rn(x2, x3);
                    const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
                    px[0][r][0] = as_u32(h0);
                    px[0][r][1] = as_u32(h1);
                    x0 -= f0.x;
                    x1 -= f0.y;
                    x2 -= f1.x;
                    x3 -= f1.y;
                    // 16 bits are left: 8 in the upper half, then 8 behind it
                    const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1), u2 = __float_as_uint(x2), u3 = __float_as_uint(x3);
                    px[1][r][0] = __byte_perm(u0, u1, 0x7632);
                    px[1][r][1] = __byte_perm(u2, u3, 0x7632);
                    x0 -= __uint_as_float(u0 & 0xffff0000u);
                    x1 -= __uint_as_float(u1 & 0xffff0000u);
                    x2 -= __uint_as_float(u2 & 0xffff0000u);
                    x3 -= __uint_as_float(u3 & 0xffff0000u);
                    px[2][r][0] = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
                    px[2][r][1] = __byte_perm(__float_as_uint(x2), __float_as_uint(x3), 0x7632);
                }
                auto code = [&](auto R, int n) {
                    constexpr int r = decltype(R)::value;
                    uint32_t c = v_codes<r>(u[n], nb[n / 4], n % 4, magic);
                    return as_u32(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&c), __floats2bfloat162_rn(144.f, 144.f)));
                };
                const std::integral_constant<int, 0> r0{};
                const std::integral_constant<int, 1> r1{};
                const std::integral_constant<int, 2> r2{};
                const std::integral_constant<int, 3> r3{};
                const uint4 v0 = make_uint4(code(r0, n0), code(r1, n0), code(r0, n1), code(r1, n1));
#pragma unroll
                for (int r = 0; r < NQ; ++r)
#pragma unroll
                    for (int i = 0; i < 3; ++i) mma_bf16(acc.o[r][2 * b], v0, px[i][r][0], px[i][r][1]);
                const uint4 v1 = make_uint4(code(r2, n0), code(r3, n0), code(r2, n1), code(r3, n1));
#pragma unroll
                for (int r = 0; r < NQ; ++r)
#pragma unroll
                    for (int i = 0; i < 3; ++i) mma_bf16(acc.o[r][2 * b + 1], v1, px[i][r][0], px[i][r][1]);
            }
        }
    }
    // the stage's next copy comes by another proxy than clear_rows' writes
    if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

constexpr size_t kRingEnd = 220 * 1024;

// Shared memory of the split kernel: query fragments of each group, the joins'
// sums, the plan, then a ring of `stages` cells per warp.
template <int NB, int TILE>
struct Smem {
    static constexpr int D = NB * 32;
    static constexpr size_t qs = (size_t)(D / 16) * 512 * (TILE == kF32W ? 2 : 1);
    static constexpr size_t all_qs = groups_of<NB, TILE>() * qs;
    static constexpr size_t comb = (size_t)warps_of<NB, TILE>() / 2 * queries_of<TILE>() * (D + 4) * 4;
    __host__ __device__ static constexpr size_t ring(int E) { return (all_qs + comb + (size_t)(E + 1) * sizeof(PlanEntry) + 127) / 128 * 128; }
};

// x g / d and x / d for 0 <= x, in 32 bits where they fit
__device__ __forceinline__ long long mul_div(long long x, int g, long long d) {
    const unsigned long long n = (unsigned long long)x * (unsigned)g;
    if (((n | (unsigned long long)d) >> 32) == 0) return (unsigned)n / (unsigned)d;
    return (long long)(n / (unsigned long long)d);
}

// A part of a range: key kk (KV head kh, slice sl) of entry e, cells [ca, cb)
// (none where the part lies in the key's setup), and the work of it.  base: the
// key's first unit of work.
struct Fragment {
    int e, kk, kh, sl, nsl, nq, c0, nc, ca, cb, keys, work;
    long long base;
};
// (inlined: as a call its struct lives in local memory, which cost 1 to 3 us a decode)
__device__ __forceinline__ void fragment_at(Fragment& f, const PlanEntry* plan, int E, int Hkv, int setup, int QPI, long long x, long long x1) {
    f.e = find_entry(plan, E, mul_div(x, 1, Hkv));
    const PlanEntry pe = plan[f.e];
    const long long first = pe.work * Hkv;
    const int len = pe.nc + setup;
    f.kk = (int)mul_div(x - first, 1, len);
    f.base = first + (long long)f.kk * len;
    const int va = (int)(x - f.base), vb = (int)min((long long)len, va + (x1 - x));
    f.work = vb - va;
    f.ca = max(0, va - setup);
    f.cb = max(0, vb - setup);
    f.nq = pe.nq;
    f.nsl = (pe.nq + QPI - 1) / QPI;
    f.kh = f.kk / f.nsl;
    f.sl = f.kk - f.kh * f.nsl;
    f.c0 = pe.c0;
    f.nc = pe.nc;
    f.keys = pe.keys;
}

// The next fragment with cells from unit x on
__device__ __forceinline__ bool next_fragment(Fragment& f, long long& x, long long x1, const SplitArgs& a, const PlanEntry* plan, int QPI) {
    while (x < x1) {
        fragment_at(f, plan, a.E, a.g.Hkv, a.setup, QPI, x, x1);
        x += f.work;
        if (f.ca < f.cb) return true;
    }
    return false;
}

// The producer side of a warp's ring: its cells (every gw-th of each fragment) in
// order.  Lanes hold the pages of its next 32 cells of the fragment.
struct Producer {
    long long x;                   // behind the fragment
    int c, cb;                     // next cell, and the fragment's end
    int row0, page, off, i;        // the lane's looked-up cell (row0 -1: none) and its bytes in the page; next lane to use
    int kh, c0, hi, listed;
    const int* table;
    const int* list;
};
// The producer enters a fragment
__device__ __forceinline__ void enter(Producer& p, const SplitArgs& a, const Fragment& n, int gwarp) {
    p.c = n.ca + gwarp;
    p.cb = n.cb;
    p.c0 = n.c0;
    p.kh = n.kh;
    int seq = n.e;
    if (a.lists) seq = n.e / a.T;
    else if (n.e >= a.n_seq) seq = a.group_start[n.e - a.n_seq];
    p.table = a.tables + (long long)seq * a.g.max_pages;
    p.listed = a.lists != nullptr;
    p.list = a.lists ? a.lists + ((long long)n.e * a.g.Hkv + n.kh) * a.keep : nullptr;
    p.hi = a.lists ? a.lens[seq] - a.T + (n.e - seq * a.T) + 1 : 0x7fffffff;
}
// Look up this warp's next 32 cells of the fragment (page numbers are checked
// where they are used, so that the load need not be waited for here)
__device__ __forceinline__ void look_up(Producer& p, const SplitArgs& a, int lane) {
    p.i = 0;
    const int cps = a.g.page_shift - 4, mask = (1 << cps) - 1;
    const int c = p.c + lane * a.gw;
    p.row0 = -1;
    if (c >= p.cb) return;
    const int at = p.listed ? c : p.c0 + c, in = at & mask;
    int slot = at >> cps;
    if (p.listed) {
        slot = p.list[slot];
        if (slot >= a.g.max_pages) atomicExch(a.g.err, kErrCounter);
        if (slot < 0 || slot >= a.g.max_pages || slot * a.g.page_rows + in * 16 >= p.hi) return;
    }
    p.row0 = slot * a.g.page_rows + in * 16;
    p.page = p.table[slot];
    p.off = (p.kh * (mask + 1) + in) * a.g.cell_bytes;
}
// On to the next fragment in which this warp has a cell; false: none
__device__ __forceinline__ bool refill(Producer& p, const SplitArgs& a, const PlanEntry* plan, int QPI, long long x1, int gwarp) {
    while (p.c >= p.cb) {
        Fragment n;
        if (!next_fragment(n, p.x, x1, a, plan, QPI)) return false;
        enter(p, a, n, gwarp);
    }
    return true;
}

// Ranges that W units of work (cells, and `setup` for each key) are cut into:
// one for each group of warps, and about a cell for each of its warps at least
// (of 1, 2, 4 and 6 cells a warp, 1 was best or near it at every size: longer
// ranges save records but leave SMs idle)
__device__ __forceinline__ int ranges(const SplitArgs& a, long long W) {
    return (int)min((long long)a.G * a.groups, (W + a.gw - 1) / a.gw);
}

// The range that holds unit x of W units of work in G ranges
__device__ __forceinline__ int range_of(long long x, int G, long long W) {
    const unsigned long long n = (unsigned long long)(x + 1) * (unsigned)G - 1;
    if (((n | (unsigned long long)W) >> 32) == 0) return (int)((unsigned)n / (unsigned)W);
    return (int)(n / (unsigned long long)W);
}

// Weight of a row's sums in its output, the sink (log2 units, -inf: none) taken in
__device__ __forceinline__ float sink_weight(float sink, float M, float L) {
    if (M == kNegInf) return 0.f;
    if (sink == kNegInf) return 1.0f / L;
    const float m = fmaxf(M, sink);
    const float al = ex2(M - m);
    return al / (L * al + ex2(sink - m));
}
__device__ __forceinline__ float sink_of(const SplitArgs& a, int h) {
    return a.sinks ? a.sinks[h] * 1.4426950408889634f : kNegInf;
}

// Four consecutive elements of an output row
__device__ __forceinline__ void store4(const SplitArgs& a, long long at, const float4& o, float w) {
    if (a.bf16)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
            make_uint2(as_u32(__floats2bfloat162_rn(o.x * w, o.y * w)), as_u32(__floats2bfloat162_rn(o.z * w, o.w * w)));
    else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(o.x * w, o.y * w, o.z * w, o.w * w);
}

// Four elements of an output row summed over the records first, first + step ..
// below last (slots of one key)
struct Sum4 {
    float M, L;
    float4 o;
};
__device__ __forceinline__ void add_sum(Sum4& s, float M, float L, const float4& o) {
    const float m = fmaxf(s.M, M);
    if (m == kNegInf) return;
    const float x = s.M == kNegInf ? 0.f : ex2(s.M - m), y = M == kNegInf ? 0.f : ex2(M - m);
    s.M = m;
    s.L = s.L * x + L * y;
    s.o.x = s.o.x * x + o.x * y;
    s.o.y = s.o.y * x + o.y * y;
    s.o.z = s.o.z * x + o.z * y;
    s.o.w = s.o.w * x + o.w * y;
}
// (kHalf: the prefix tiles' records, fp16 times a power of two)
template <int D, bool kHalf = false>
__device__ __forceinline__ void add_records(const SplitArgs& a, Sum4& s, long long slot0, int first, int last, int step, int row, int col) {
    constexpr int U = 8;                               // records in flight
    for (int r0 = first; r0 < last; r0 += U * step) {
        float2 ml[U];
        float back[U];
        float4 o[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            ml[i] = make_float2(kNegInf, 0.f);
            back[i] = 1.f;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r0 + i * step < last) {
                const long long at = (slot0 + r0 + i * step) * (kHalf ? a.tile_rows : a.rec_rows) + row;
                if constexpr (kHalf) {
                    const float4 x4 = __ldcg(reinterpret_cast<const float4*>(a.part2_ml) + at);
                    ml[i] = make_float2(x4.x, x4.y);
                    back[i] = x4.z;
                    const uint2 h = __ldcg(reinterpret_cast<const uint2*>(a.part2_o + at * D + col));
                    const float2 x = __half22float2(as_h2(h.x)), y = __half22float2(as_h2(h.y));
                    o[i] = make_float4(x.x, x.y, y.x, y.y);
                } else {
                    ml[i] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at);
                    o[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + col));
                }
            }
        }
        float m = s.M;
#pragma unroll
        for (int i = 0; i < U; ++i) m = fmaxf(m, ml[i].x);
        if (m == kNegInf) continue;
        const float al = s.M == kNegInf ? 0.f : ex2(s.M - m);
        s.M = m;
        s.L *= al;
        s.o.x *= al; s.o.y *= al; s.o.z *= al; s.o.w *= al;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float w = ml[i].x == kNegInf ? 0.f : ex2(ml[i].x - m);
            s.L = fmaf(ml[i].y, w, s.L);
            const float v = kHalf ? back[i] * w : w;
            s.o.x = fmaf(o[i].x, v, s.o.x);
            s.o.y = fmaf(o[i].y, v, s.o.y);
            s.o.z = fmaf(o[i].z, v, s.o.z);
            s.o.w = fmaf(o[i].w, v, s.o.w);
        }
    }
}

template <int NB, bool F8, int TILE>
__global__ void __launch_bounds__(warps_of<NB, TILE>() * 32, 1) split_kernel(const __grid_constant__ SplitArgs a, const int stages) {
    constexpr int D = NB * 32, D4 = D / 4;
    constexpr int kWarps = warps_of<NB, TILE>(), kThreads = kWarps * 32;
    constexpr bool HL = two_parts<TILE>();
    constexpr int QPI = queries_of<TILE>(), NQ = QPI / 8;
    constexpr int CELL = NB * (F8 ? 1024 : 928);
    constexpr int PAD = D + 4;                        // row stride of the joins' sums: lanes of a store in different banks
    using S = Smem<NB, TILE>;
    extern __shared__ __align__(128) uint8_t smem[];
    PlanEntry* plan = reinterpret_cast<PlanEntry*>(smem + S::all_qs + S::comb);
    __shared__ RowInfo s_ri[groups_of<NB, TILE>()];
    __shared__ float s_m[kWarps][16], s_l[kWarps][16];
    __shared__ long long s_wsum[kWarps];
    __shared__ int s_ksum[kWarps];
    __shared__ int s_row0[kWarps][kMaxStages];        // first row of the cell in a stage, -1: none
    __shared__ __align__(8) uint64_t s_bar[kWarps][kMaxStages];
    __shared__ int s_abort, s_last[groups_of<NB, TILE>()];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (lane < stages) dev::mbar_init(dev::smem_u32(&s_bar[warp][lane]), 1);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // ---- the CTA's groups of gw warps work on ranges of their own: while one
    // group joins and changes keys (some 5 us of latencies) the others compute
    const int gw = a.gw, group = warp / gw, gwarp = warp - group * gw, gtid = tid - group * gw * 32;
    const int range = group * gridDim.x + blockIdx.x;
    uint8_t* qs = smem + group * S::qs;
    float* comb = reinterpret_cast<float*>(smem + S::all_qs) + (size_t)group * (gw / 2) * QPI * PAD;
    RowInfo& ri = s_ri[group];
    auto sync_group = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gw * 32) : "memory"); };
    const uint32_t ring = dev::smem_u32(smem) + (uint32_t)S::ring(a.E) + (uint32_t)(warp * stages * CELL);
    uint8_t* ring_p = smem + S::ring(a.E) + (size_t)warp * stages * CELL;
    const uint32_t bar0 = dev::smem_u32(&s_bar[warp][0]);

    // ---- queries: a warp takes every gw-th query row of the fragment, loads it
    // into registers and later lays it out as A fragments in shared memory
    constexpr int RPW = QPI / 4;                       // rows of a warp at most
    float qv[RPW][NB];
    Query qq[RPW];
    auto load_queries = [&](const Fragment& f) {
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
            const int r = gwarp + i * gw, qi = f.sl * QPI + r;
            qq[i] = Query{0, 0, 0, 0, -1};
            const bool valid = r < QPI && qi < f.nq;
            if (valid) qq[i] = query_of(a, plan[f.e], f.e, f.kh, qi);
            const long long at = (((long long)qq[i].seq * a.T + qq[i].t) * a.Hq + qq[i].h) * D + lane;
#pragma unroll
            for (int b = 0; b < NB; ++b) qv[i][b] = valid ? load_q(a.q, at + 32 * b, a.bf16) : 0.f;
        }
    };
    auto place_queries = [&]() {
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
            const int r = gwarp + i * gw;
            if (r >= QPI) break;
            uint32_t am = 0u;                              // bits of the largest |element|: NaN above infinity
#pragma unroll
            for (int b = 0; b < NB; ++b) am = max(am, __float_as_uint(qv[i][b]) & 0x7fffffffu);
            am = __reduce_max_sync(0xffffffffu, am);
            const bool bad = am >= kInfBits;
            // scaled by a power of two to a largest element in [512, 1024)
            const int ex = am > 0u && !bad ? min(max((int)(am >> 23) - 127 - 9, -117), 118) : 0;
            const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (lane == 0) {
                ri.fac[r] = factor(a.qscale * __uint_as_float((uint32_t)(127 + ex) << 23));
                ri.lo[r] = qq[i].lo;
                ri.hi[r] = qq[i].hi;
                ri.bad[r] = bad;
            }
            const int wi = lane & 7, j = lane >> 3;
            const int reg = ((wi & 3) >> 1) * 2, half = wi & 1;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float y = bad ? 0.f : qv[i][b] * up;
                const __half hi = __float2half_rn(y);
                const int at = ((HL ? (r >> 3) * 2 * NB : 0) + 2 * b + (wi >> 2)) * 32 + 4 * (r & 7) + j;
                __half* dst = reinterpret_cast<__half*>(qs + at * 16);
                if (TILE == kT8) {                         // (rows 8 .. 15 of the tile are zeros)
                    dst[2 * reg + half] = hi;
                    dst[2 * (reg + 1) + half] = __float2half_rn(0.f);
                } else if (HL) {
                    dst[2 * reg + half] = hi;
                    dst[2 * (reg + 1) + half] = __float2half_rn(y - __half2float(hi));
                } else {
                    dst[2 * (reg + (r >> 3)) + half] = hi;
                }
            }
        }
    };
    long long W = 0, x = 0, x1 = 0;
    int G = 1;
    Fragment f{};
    Producer pr;
    pr.c = pr.cb = 0;
    pr.row0 = -1;
    pr.i = 32;
    const uint64_t policy = dev::evict_first_policy();      // a decode reads each cell once, or nearly
    auto produce = [&](int st) {                           // the next cell of the ring, into stage st
        if (pr.c >= pr.cb) {
            if (!refill(pr, a, plan, QPI, x1, gwarp)) return;
            pr.i = 32;
        }
        if (pr.i == 32) look_up(pr, a, lane);
        if (lane == pr.i) {
            const uint32_t bar = bar0 + 8u * st;
            const bool there = pr.row0 >= 0 && pr.page >= 0 && pr.page < a.g.n_pages;
            if (pr.row0 >= 0 && !there) atomicExch(a.g.err, kErrCounter);
            s_row0[warp][st] = there ? pr.row0 : -1;
            if (there) {
                dev::mbar_expect_tx(bar, CELL);
                asm volatile(
                    "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                    ::"r"(ring + (uint32_t)(st * CELL)), "l"(a.g.pool + pr.page * a.g.page_bytes + pr.off), "r"(CELL), "r"(bar), "l"(policy)
                    : "memory");
            } else {
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
            }
        }
        ++pr.i;
        pr.c += a.gw;
    };

    float zero[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.f32 %0, 0f00000000;" : "=f"(zero[i]));
    const uint32_t magic = held(HL ? 0x43004300u : 0x64006400u);   // 128 in bf16, 1024 in fp16: codes in the low bits add to it
    const uint32_t exps = held(0x64646464u);
    int st = 0;
    uint32_t phase = 0;
    // (After the tile kernel too: that waited for what came before, but only a grid's
    // own wait makes earlier grids' writes visible to it.)
    wait_for_earlier();
    // ---- the plan: prefix sums of the entries' work (one warp's scan for up to
    // 32 entries, else every thread's share and a scan over the CTA)
    {
        const int per = (a.E + kThreads - 1) / kThreads;
        const bool one_warp = a.E <= 32;
        long long w = 0;
        int k = 0;
        if (!one_warp || warp == 0) {
            for (int i = 0; i < per; ++i) {
                const int e = tid * per + i;
                if (e < a.E) {
                    const EntryWork ew = entry_work(a, e, blockIdx.x == 0);
                    const int sl = (ew.nq + QPI - 1) / QPI;
                    plan[e].nc = ew.nc;
                    plan[e].c0 = ew.c0;
                    plan[e].nq = ew.nq;
                    plan[e].rows = ew.rows;
                    plan[e].lo = ew.lo;
                    plan[e].work = w;
                    plan[e].keys = k;
                    w += ew.nc ? (long long)(ew.nc + a.setup) * sl : 0;
                    k += sl;
                }
            }
        }
        long long wi = w;
        int ki = k;
        if (!one_warp || warp == 0) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, wi, o);
                const int z = __shfl_up_sync(0xffffffffu, ki, o);
                if (lane >= o) {
                    wi += y;
                    ki += z;
                }
            }
        }
        long long wb = wi - w;
        int kb = ki - k;
        if (!one_warp) {
            if (lane == 31) {
                s_wsum[warp] = wi;
                s_ksum[warp] = ki;
            }
            __syncthreads();
            for (int i = 0; i < warp; ++i) {
                wb += s_wsum[i];
                kb += s_ksum[i];
            }
        }
        if (!one_warp || warp == 0) {
            for (int i = 0; i < per; ++i) {
                const int e = tid * per + i;
                if (e < a.E) {
                    plan[e].work += wb;
                    plan[e].keys += kb;
                }
            }
            if (tid == (one_warp ? 31 : kThreads - 1)) {
                // groups that overlap could ask for more records than there are
                const bool fits = (long long)(kb + k) * a.g.Hkv <= a.max_keys;
                if (!fits) atomicExch(a.g.err, kErrCounter);
                plan[a.E].work = fits ? wb + w : 0;
                plan[a.E].keys = kb + k;
                plan[a.E].nc = plan[a.E].c0 = plan[a.E].nq = plan[a.E].rows = plan[a.E].lo = 0;
            }
        }
        __syncthreads();
        if (!a.fuse && blockIdx.x == 0)
            for (int e = tid; e <= a.E; e += kThreads) a.plan[e] = plan[e];
    }
    let_next_start();
    W = plan[a.E].work * a.g.Hkv;
    G = ranges(a, W);
    if (a.fuse) {
        // entries without rows have no key: their outputs are zeros
        for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
            if (plan[e].nc != 0 && W != 0) continue;
            const long long n = (long long)(a.lists ? 1 : a.T) * a.Hq * D, at = e * n;
            for (long long i = 4 * tid; i < n; i += 4 * kThreads) store4(a, at + i, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
        }
    }
    if (range >= G) return;
    x = mul_div(W, range, G);
    x1 = mul_div(W, range + 1, G);
    if (!next_fragment(f, x, x1, a, plan, QPI)) return;
    pr.x = x;
    enter(pr, a, f, gwarp);
    look_up(pr, a, lane);
    for (int pass = 0;; ++pass) {
        // one cell a warp, then the queries, then the other stages: query loads
        // behind the whole first burst of copies would take 3 us
        load_queries(f);
        if (pass > 0) sync_group();                        // the last fragment's sums and queries are free
#pragma unroll 1
        for (int s = 0; s < (pass == 0 ? stages : 1); ++s) {
            if (pass == 0) produce(s);
            if (s == 0) place_queries();
        }
        sync_group();
        const int g = lane >> 2, j = lane & 3;
        Acc<NB, F8, TILE> acc;
        LaneRows<NQ> lr;
        {
            const bool v = lane < QPI && f.sl * QPI + lane < f.nq;
            const int lo = v ? ri.lo[lane] : 0, hi = v ? ri.hi[lane] : 0;
            const bool some = v && hi > lo;
            lr.lo_max = __reduce_max_sync(0xffffffffu, v ? lo : 0);
            lr.hi_min = __reduce_min_sync(0xffffffffu, v ? hi : 0x7fffffff);
            lr.lo_min = __reduce_min_sync(0xffffffffu, some ? lo : 0x7fffffff);
            lr.hi_max = __reduce_max_sync(0xffffffffu, some ? hi : 0);
        }
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            acc.m[r] = kNone;
            acc.l[r] = 0.f;
            lr.fac[r] = ri.fac[g + 8 * r];
            lr.lo[r] = ri.lo[g + 8 * r];
            lr.hi[r] = ri.hi[g + 8 * r];
#pragma unroll
            for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc.o[r][n][i] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < NQ; ++r)
#pragma unroll
            for (int b = 0; b < (HL && !F8 ? NB : 1); ++b) acc.mt[r][b] = 0.f;

        // ---- its cells, warp by warp
        for (int c = f.ca + gwarp; c < f.cb; c += gw) {
            const bool there = wait_bounded(bar0 + 8u * st, phase, &s_abort, a.g.err);
            const int row0 = s_row0[warp][st];
            if (there && row0 >= 0 && row0 < lr.hi_max)
                take_cell<NB, F8, TILE>(a, ring_p + st * CELL, row0, qs, lr, lane, zero, magic, exps, acc);
            __syncwarp();
            if (there) produce(st);
            if (++st == stages) {
                st = 0;
                phase ^= 1u;
            }
        }

        // ---- join the group's warps: a common reference, the upper warps' sums
        // onto the lower half's (12 warps: 4 onto 4 first), then every thread
        // adds up its elements over what is left
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], 1);
            acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], 2);
            if (j == 0) {
                s_m[warp][g + 8 * r] = acc.m[r];
                s_l[warp][g + 8 * r] = acc.l[r];
            }
        }
        if constexpr (HL && !F8) {
#pragma unroll
            for (int r = 0; r < NQ; ++r)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float t = acc.mt[r][b];
                    t += __shfl_xor_sync(0xffffffffu, t, 1);
                    t += __shfl_xor_sync(0xffffffffu, t, 2);
                    const float t0 = __shfl_sync(0xffffffffu, t, 8 * j), t1 = __shfl_sync(0xffffffffu, t, 8 * j + 4);
#pragma unroll
                    for (int rp = 0; rp < 2; ++rp) {
                        acc.o[r][2 * b + rp][0] += t0;
                        acc.o[r][2 * b + rp][1] += t1;
                        acc.o[r][2 * b + rp][2] += t0;
                        acc.o[r][2 * b + rp][3] += t1;
                    }
                }
        }
        sync_group();
        const int w0 = warp - gwarp;
        auto group_max = [&](int row) {
            float m = kNone;
#pragma unroll 4
            for (int w = w0; w < w0 + gw; ++w) m = fmaxf(m, s_m[w][row]);
            return m;
        };
#pragma unroll
        for (int r = 0; r < NQ; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 2 * j + i + 8 * r;
                const float fa = ex2(s_m[warp][row] - group_max(row));
#pragma unroll
                for (int n = 0; n < 2 * NB; ++n) {
                    acc.o[r][n][i] *= fa;
                    acc.o[r][n][2 + i] *= fa;
                }
            }
        const int rows = min(QPI, f.nq - f.sl * QPI);
        auto region = [&](int w, auto&& body) {            // the lane's four-element pieces in region w
            float* base = comb + (size_t)w * QPI * PAD + 4 * g;
#pragma unroll
            for (int r = 0; r < NQ; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = 2 * j + i + 8 * r;
                    if (row >= rows) continue;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        body(reinterpret_cast<float4*>(base + row * PAD + 32 * b), acc.o[r][2 * b][i], acc.o[r][2 * b][2 + i],
                             acc.o[r][2 * b + 1][i], acc.o[r][2 * b + 1][2 + i]);
                }
        };
        auto put = [](float4* p, float& x, float& y, float& z, float& w) { *p = make_float4(x, y, z, w); };
        auto add = [](float4* p, float& x, float& y, float& z, float& w) {
            const float4 v = *p;
            x += v.x; y += v.y; z += v.z; w += v.w;
        };
        const int n0 = gw & (gw - 1) ? 4 : gw / 2;
        for (int lo = gw - 2 * n0; lo >= 0; lo -= n0) {
            if (gwarp >= lo + n0 && gwarp < lo + 2 * n0) region(gwarp & (n0 - 1), put);
            sync_group();
            if (gwarp >= lo && gwarp < lo + n0) region(gwarp & (n0 - 1), add);
            if (lo > 0) sync_group();
        }
        if (gwarp < n0) region(gwarp, put);                // the region that only this warp read
        sync_group();

        const int rec0 = range_of(f.base + a.setup, G, W), n_rec = range_of(f.base + a.setup + f.nc - 1, G, W) - rec0 + 1;
        const long long key = (long long)f.keys * a.g.Hkv + f.kk;
        const bool whole = a.fuse && n_rec == 1;
        for (int c = gtid; c < rows * D4; c += gw * 32) {
            const int row = c / D4, col = 4 * (c % D4);
            float4 o = *reinterpret_cast<const float4*>(comb + row * PAD + col);
            for (int w = 1; w < n0; ++w) {
                const float4 y = *reinterpret_cast<const float4*>(comb + (size_t)w * QPI * PAD + row * PAD + col);
                o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
            }
            const float m = group_max(row);
            float l = 0.f;
#pragma unroll 4
            for (int w = w0; w < w0 + gw; ++w) l = fmaf(s_l[w][row], ex2(s_m[w][row] - m), l);
            const float M = settle(l, m, ri.bad[row]) ? m - kShift : kNegInf;
            if (whole) {
                const Query q = query_of(a, plan[f.e], f.e, f.kh, f.sl * QPI + row);
                store4(a, (((long long)q.seq * a.T + q.t) * a.Hq + q.h) * D + col, o, sink_weight(sink_of(a, q.h), M, l));
            } else {
                const long long at = (range + key) * a.rec_rows + row;
                *reinterpret_cast<float4*>(a.part_o + at * D + col) = o;
                if (col == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(M, l);
            }
        }
        if (a.fuse && !whole) {
            // the group that completes a key's records joins them; the others go on
            __threadfence();
            sync_group();
            if (gtid == 0) {
                const bool last = atomicAdd(a.arrived + key, 1) == n_rec - 1;
                if (last) a.arrived[key] = 0;
                s_last[group] = last;
                __threadfence();
            }
            sync_group();
            if (s_last[group]) {
                // threads in `sets` that share the records, then one of each adds them up
                const int n = rows * D4;
                int sets = 1;
                while (2 * sets * n <= gw * 32 && 2 * sets <= n_rec && 2 * sets <= gw / 2) sets *= 2;
                for (int c0 = 0; c0 < n; c0 += gw * 32) {
                    const int set = sets > 1 ? gtid / n : 0, c = sets > 1 ? gtid - set * n : c0 + gtid;
                    const int row = c / D4, col = 4 * (c % D4);
                    const bool on = set < sets && c < n;
                    Query q{0, 0, 0, 0, 0};
                    float sink = kNegInf;
                    Sum4 s{kNegInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
                    if (on) {
                        q = query_of(a, plan[f.e], f.e, f.kh, f.sl * QPI + row);
                        sink = sink_of(a, q.h);
                        add_records<D>(a, s, rec0 + key, set, n_rec, sets, row, col);
                    }
                    if (sets > 1) {
                        float* p = comb + (size_t)set * QPI * PAD;
                        if (on && set > 0) {
                            *reinterpret_cast<float4*>(p + row * PAD + col) = s.o;
                            if (col == 0) {
                                s_m[w0 + set][row] = s.M;
                                s_l[w0 + set][row] = s.L;
                            }
                        }
                        sync_group();
                        if (on && set == 0)
                            for (int w = 1; w < sets; ++w)
                                add_sum(s, s_m[w0 + w][row], s_l[w0 + w][row], *reinterpret_cast<const float4*>(p + (size_t)w * QPI * PAD + row * PAD + col));
                    }
                    if (on && set == 0)
                        store4(a, (((long long)q.seq * a.T + q.t) * a.Hq + q.h) * D + col, s.o, sink_weight(sink, s.M, s.L));
                }
            }
        }
        if (!next_fragment(f, x, x1, a, plan, QPI)) break;
    }
    if (s_abort) {                                         // a wait ran out: let copies in flight land before the CTA ends
        const long long t0 = clock64();
        while (clock64() - t0 < (1LL << 30)) __nanosleep(1000);
    }
}

// ------------------------------------------------------------ merge kernel

// Outputs of a shared decode: D / 4 threads a row (sequence, t, head), over the
// records of its own rows' key and of its group's prefix, and the sink.
template <int NB>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ SplitArgs a, int QPI) {
    constexpr int D = NB * 32, D4 = D / 4;
    wait_for_earlier();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = i / D4;
    const int col = 4 * (int)(i % D4);
    if (row >= (long long)a.n_seq * a.T * a.Hq) return;
    const int h = (int)(row % a.Hq), st = (int)(row / a.Hq);
    const int seq = st / a.T, t = st - seq * a.T;
    const int kh = h / a.hpk, hr = h - kh * a.hpk;
    const float sink = sink_of(a, h);
    const long long W = a.plan[a.E].work * a.g.Hkv;
    const int G = ranges(a, W);
    Sum4 s{kNegInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    auto fold = [&](int e, int qi) {
        const PlanEntry pe = a.plan[e];
        if (pe.nc == 0 || W == 0) return;
        const int nsl = (pe.nq + QPI - 1) / QPI;
        const int kk = kh * nsl + qi / QPI;
        const long long xa = pe.work * a.g.Hkv + (long long)kk * (pe.nc + a.setup) + a.setup;
        const int c0 = range_of(xa, G, W), c1 = range_of(xa + pe.nc - 1, G, W);
        add_records<D>(a, s, (long long)pe.keys * a.g.Hkv + kk + c0, 0, c1 - c0 + 1, 1, qi % QPI, col);
    };
    fold(seq, t * a.hpk + hr);
    const int grp = group_of(a, seq);
    if (grp >= 0) {
        int gs, ge;
        members(a, grp, gs, ge);
        const int qi = ((seq - gs) * a.T + t) * a.hpk + hr;
        if (seq >= gs && seq < ge) {
            if (tile_group(a, (ge - gs) * a.hpk * a.T)) {
                const long long W2 = a.plan2[a.n_groups].work * a.g.Hkv;
                const PlanEntry pe = a.plan2[grp];
                if (pe.nc != 0 && W2 != 0) {
                    const int G2 = (int)min((long long)a.G, W2), nqb = (pe.nq + a.tile_rows - 1) / a.tile_rows;
                    const int kk = kh * nqb + qi / a.tile_rows;
                    const long long xa = pe.work * a.g.Hkv + (long long)kk * pe.nc;
                    const int c0 = range_of(xa, G2, W2), c1 = range_of(xa + pe.nc - 1, G2, W2);
                    add_records<D, true>(a, s, (long long)pe.keys * a.g.Hkv + kk + c0, 0, c1 - c0 + 1, 1, qi % a.tile_rows, col);
                }
            } else {
                fold(a.n_seq + grp, qi);
            }
        }
    }
    store4(a, row * D + col, s.o, sink_weight(sink, s.M, s.L));
}

template <int NB, bool F8, int TILE>
cudaError_t launch_split_t(const SplitArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(split_kernel<NB, F8, TILE>, done, true);
    if (e != cudaSuccess) return e;
    using S = Smem<NB, TILE>;
    constexpr size_t cells = (size_t)warps_of<NB, TILE>() * NB * (F8 ? 1024 : 928);
    // the ring takes what the plan leaves of 220 KB: a cell for each warp at least
    static_assert(S::ring(kMaxEntries) + cells <= kRingEnd, "no room for the cells");
    if (a.E > kMaxEntries) return cudaErrorInvalidValue;
    const int stages = (int)std::min<size_t>(kMaxStages, (kRingEnd - S::ring(a.E)) / cells);
    return launch_dependent(split_kernel<NB, F8, TILE>, dim3((unsigned)a.G), warps_of<NB, TILE>() * 32,
                            S::ring(a.E) + stages * cells, s, a, stages);
}

template <int NB, bool F8>
cudaError_t launch_split_f(const SplitArgs& a, cudaStream_t s) {
    if constexpr (NB < 8)
        if (!a.bf16 && a.tile == 16) return launch_split_t<NB, F8, kF32W>(a, s);
    if (!a.bf16) return launch_split_t<NB, F8, kF32>(a, s);
    return a.tile == 8 ? launch_split_t<NB, F8, kT8>(a, s) : launch_split_t<NB, F8, kT16>(a, s);
}

template <int NB>
cudaError_t launch_split_nb(const SplitArgs& a, cudaStream_t s) {
    return a.g.fp8 ? launch_split_f<NB, true>(a, s) : launch_split_f<NB, false>(a, s);
}

}  // namespace

// f32 queries of head_dim 256 stay at 8: two parts of 16 leave few registers and
// stages (16k rows, 4 KV heads of 8 x 4 queries, P d in two parts: 43 us, 8: 38),
// where smaller heads gain (8 sequences of 16k rows, 8 KV heads of 128, 16 queries:
// 102 us, 8: 119)
int split_tile(int NB, bool bf16, int most_queries) { return most_queries > 8 && (bf16 || NB < 8) ? 16 : 8; }

int split_warps(int NB, int tile) {
    if (tile == 16) return NB == 2 ? warps_of<2, kT16>() : NB == 4 ? warps_of<4, kT16>() : warps_of<8, kT16>();
    return NB == 2 ? warps_of<2, kT8>() : NB == 4 ? warps_of<4, kT8>() : warps_of<8, kT8>();
}
static_assert(warps_of<2, kT8>() == warps_of<2, kF32>() && warps_of<4, kT8>() == warps_of<4, kF32>() &&
              warps_of<8, kT8>() == warps_of<8, kF32>() && warps_of<2, kT16>() == warps_of<2, kF32W>() &&
              warps_of<4, kT16>() == warps_of<4, kF32W>(),
              "tiles of as many queries share a CTA size");

cudaError_t launch_split(const SplitArgs& a, cudaStream_t s) {
    switch (a.g.NB()) {
        case 2: return launch_split_nb<2>(a, s);
        case 4: return launch_split_nb<4>(a, s);
        default: return launch_split_nb<8>(a, s);
    }
}

cudaError_t launch_merge(const SplitArgs& a, cudaStream_t s) {
    const long long rows = (long long)a.n_seq * a.T * a.Hq;
    const dim3 grid((unsigned)((rows * (a.g.D / 4) + 255) / 256));
    switch (a.g.NB()) {
        case 2: return launch_dependent(merge_kernel<2>, grid, 256, 0, s, a, a.tile);
        case 4: return launch_dependent(merge_kernel<4>, grid, 256, 0, s, a, a.tile);
        default: return launch_dependent(merge_kernel<8>, grid, 256, 0, s, a, a.tile);
    }
}

}  // namespace paged
}  // namespace kvq
