// Decode attention over the paged cache: dense, with a shared prefix, or over
// listed pages.
//
// Mathematics.  For each query, o = sum_t p_t v_t / sum_t p_t with
// p_t = 2^(s_t - m), s_t the scaled score in log2 units and m a reference that
// only moves when a score passes it by 8 (one pass over the rows).  Rows come in
// cells of 16 rows of one KV head; a warp takes a cell at a time and multiplies
// 16 query rows with it on the tensor cores (mma.m16n8k16): S = Q K^T and
// O += P V.  The cell layout is the operands' register layout, so a lane's
// loads are its fragments: K and V bytes turn into fp16 pairs in registers,
// two codes an instruction, and nothing passes through shared memory.
//   K: codes are small integers, exact in fp16, so the products with the query
//      run on codes and each 32-element block's sum is scaled by its d in f32.
//   V: v = u d + m in one half2 fma a pair of rows (one rounding to fp16).
// f32 queries (HL) keep f32 accuracy with 8 queries a tile: rows 0..7 of the A
// operand carry the high part and rows 8..15 the low part of the same numbers.
// For Q these are two fp16 (22 bits of a query scaled to its largest element);
// for P d two bf16 (16 bits, any range) against the exact codes u - 16, with
// sum p (m + 16 d) kept in f32 beside it.
//
// Why tensor cores for one token: a query-row tile costs the same for 1 or 16
// queries, and the work that grows with the bytes is only the unpacking, about
// 4.5 instructions a warp-element pair of K and V, where the multiply-add form
// needs as many again for each 4 queries.
//
// Work is cut stream-K fashion: see kvq_paged.cuh.
#include "kvq_device.cuh"
#include "kvq_paged.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

namespace kvq {
namespace paged {
namespace {

using dev::kLazy;
using dev::kNegInf;
constexpr float kShift = 6.0f;         // p is held as 2^6 p: fp16 keeps 2^-20 of the largest in full
constexpr int kMaxStages = 8;
constexpr int kCombine = 4;            // warps' sums that the join holds at once

// Warps of a CTA (one CTA an SM): as many as the accumulators leave registers
// for; 12 of 168 registers at head_dim 128.
template <int NB>
constexpr int warps_of() { return NB == 2 ? 16 : NB == 4 ? 12 : 8; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// code bytes (biased by 128) sel of w under the exponent of 1024, minus 1152: exact
__device__ __forceinline__ uint32_t k_pair(uint32_t w, uint32_t sel) {
    return as_u32(__hsub2(as_h2(__byte_perm(w, 0x64646464u, sel)), as_h2(0x64806480u)));
}
// two E4M3 bytes as a half pair, exact
__device__ __forceinline__ uint32_t f8_pair(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The 5-bit codes of element r of two rows, in the low bits of each half word
template <int R>
__device__ __forceinline__ uint32_t v_codes(uint32_t unit, uint32_t nib, int n4, uint32_t magic) {
    if constexpr (R == 0) return (unit & 0x001f001fu) | magic;
    else if constexpr (R == 1) return ((unit >> 5) & 0x001f001fu) | magic;
    else if constexpr (R == 2) return ((unit >> 10) & 0x001f001fu) | magic;
    else return (((unit >> 11) & 0x00100010u) | magic) | ((nib >> (4 * n4)) & 0x000f000fu);
}

// ------------------------------------------------------------ work entries

__device__ __forceinline__ bool len_ok(const SplitArgs& a, int len) {
    return len >= 0 && len <= (long long)a.g.max_pages << a.g.page_shift;
}

// group of a sequence (-1: none)
__device__ __forceinline__ int group_of(const SplitArgs& a, int seq) {
    if (a.n_groups == 0 || seq < a.group_start[0] || seq >= a.group_start[a.n_groups]) return -1;
    int lo = 0, hi = a.n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.group_start[mid] <= seq) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int prefix_rows(const SplitArgs& a, int grp) {
    const int p = a.prefix_len[grp];
    return len_ok(a, p) ? p : 0;
}

// members of a group, [gs, ge); none if its bounds are out of order
__device__ __forceinline__ void members(const SplitArgs& a, int grp, int& gs, int& ge) {
    gs = a.group_start[grp];
    ge = a.group_start[grp + 1];
    if (gs < 0 || ge > a.n_seq || ge < gs) gs = ge = 0;
}

struct EntryWork {
    int nc, c0, nq;
};

__device__ __forceinline__ EntryWork entry_work(const SplitArgs& a, int e, bool report) {
    EntryWork w{0, 0, 0};
    int lo = 0, hi = 0;
    if (a.lists) {
        const int seq = e / a.T, t = e - seq * a.T;
        const int len = a.lens[seq];
        if (!len_ok(a, len)) {
            if (report) atomicExch(a.g.err, kErrCounter);
            return w;
        }
        w.nq = a.hpk;
        if (len - a.T + t >= 0) w.nc = a.keep * a.g.cells_per_page();
        return w;
    }
    if (e < a.n_seq) {
        const int len = a.lens[e];
        if (!len_ok(a, len)) {
            if (report) atomicExch(a.g.err, kErrCounter);
            return w;
        }
        w.nq = a.hpk * a.T;
        hi = len;
        lo = a.window > 0 ? max(0, len - a.T + 1 - a.window) : 0;
        const int grp = group_of(a, e);
        if (grp >= 0) lo = max(lo, prefix_rows(a, grp));
    } else {
        const int grp = e - a.n_seq;
        int gs, ge;
        members(a, grp, gs, ge);
        if (report && (a.group_start[grp + 1] < a.group_start[grp] || a.group_start[grp] < 0 ||
                       a.group_start[grp + 1] > a.n_seq || !len_ok(a, a.prefix_len[grp])))
            atomicExch(a.g.err, kErrCounter);
        w.nq = (ge - gs) * a.hpk * a.T;
        hi = prefix_rows(a, grp);
        lo = 0;
        if (a.window > 0) {                       // rows before every member's window are not read
            lo = hi;
            for (int m = gs; m < ge; ++m) lo = min(lo, max(0, a.lens[m] - a.T + 1 - a.window));
        }
        if (ge == gs) hi = lo;
    }
    if (hi > lo) {
        w.c0 = lo >> 4;
        w.nc = ((hi + 15) >> 4) - w.c0;
    }
    return w;
}

// Query row qi of an entry for KV head g: sequence, row t and head; and the
// rows it sees, [lo, hi) (hi <= lo: none).
struct Query {
    int seq, t, h, lo, hi;
};
__device__ __forceinline__ Query query_of(const SplitArgs& a, int e, int g, int qi) {
    Query q;
    int within = qi;
    const int Qh = a.hpk * a.T;
    if (a.lists) {
        q.seq = e / a.T;
        q.t = e - q.seq * a.T;
    } else {
        q.seq = e;
        if (e >= a.n_seq) {
            const int m = qi / Qh;
            q.seq = a.group_start[e - a.n_seq] + m;
            within = qi - m * Qh;
        }
        q.t = within / a.hpk;
        within -= q.t * a.hpk;
    }
    q.h = g * a.hpk + within;
    const int len = a.lens[q.seq];
    q.hi = len_ok(a, len) ? len - a.T + q.t + 1 : 0;
    q.lo = a.window > 0 ? max(0, q.hi - a.window) : 0;
    if (!a.lists) {
        if (e >= a.n_seq) q.hi = min(q.hi, prefix_rows(a, e - a.n_seq));
        else if (a.n_groups) {
            const int grp = group_of(a, e);
            if (grp >= 0) q.lo = max(q.lo, prefix_rows(a, grp));
        }
    }
    return q;
}

// largest e with plan[e].work <= x (x below the total)
__device__ __forceinline__ int find_entry(const PlanEntry* plan, int E, long long x) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (plan[mid].work <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float load_q(const void* q, long long idx, int bf16) {
    if (bf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[idx]);
    return reinterpret_cast<const float*>(q)[idx];
}

// ------------------------------------------------------------ split kernel

template <int NB, bool F8, bool HL>
struct Acc {
    float o[4 * NB][4];        // n-tile 4b + r: element 32b + 8j + r (cols 0) and + 4 (cols 1)
    float m[2], l[2];          // rows g and g + 8 (HL: row g)
    float mt[HL && !F8 ? NB : 1];
};

struct RowInfo {
    float fac[16];
    int lo[16], hi[16];
    int lo_min, lo_max, hi_min, hi_max;
};

// One cell: 16 rows from logical row row0 on, into the warp's accumulators
template <int NB, bool F8, bool HL>
__device__ __forceinline__ void take_cell(const SplitArgs& a, const uint8_t* __restrict__ cell, int row0,
                                          const uint4* __restrict__ qs, const RowInfo& ri, int lane,
                                          Acc<NB, F8, HL>& acc) {
    const int g = lane >> 2, j = lane & 3;
    // ---- scores
    float sc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[t][i] = 0.f;
#pragma unroll
    for (int bp = 0; bp < NB / 2; ++bp) {
        uint4 kk[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) kk[t] = *reinterpret_cast<const uint4*>(cell + bp * 1024 + t * 512 + lane * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int b = 2 * bp + e;
            const uint4 a0 = qs[(2 * b) * 32 + lane], a1 = qs[(2 * b + 1) * 32 + lane];
            if constexpr (F8) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t w0 = e ? kk[t].z : kk[t].x, w1 = e ? kk[t].w : kk[t].y;
                    mma_f16(sc[t], a0, f8_pair(w0), f8_pair(w0 >> 16));
                    mma_f16(sc[t], a1, f8_pair(w1), f8_pair(w1 >> 16));
                }
            } else {
                const uint2 ks = *reinterpret_cast<const uint2*>(cell + 512 * NB + (j * NB + b) * 8);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t w0 = e ? kk[t].z : kk[t].x, w1 = e ? kk[t].w : kk[t].y;
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(c, a0, k_pair(w0, 0x4140u), k_pair(w0, 0x4342u));
                    mma_f16(c, a1, k_pair(w1, 0x4140u), k_pair(w1, 0x4342u));
                    const float2 d = __half22float2(as_h2(t ? ks.y : ks.x));
                    sc[t][0] = fmaf(c[0], d.x, sc[t][0]);
                    sc[t][1] = fmaf(c[1], d.y, sc[t][1]);
                    sc[t][2] = fmaf(c[2], d.x, sc[t][2]);
                    sc[t][3] = fmaf(c[3], d.y, sc[t][3]);
                }
            }
        }
    }
    // ---- scale, cap, mask; the reference maximum
    constexpr int NR = HL ? 1 : 2;
    const bool edge = row0 < ri.lo_max || row0 + 16 > ri.hi_min;
    bool move = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const float f = ri.fac[g + 8 * r];
        const int lo = ri.lo[g + 8 * r], hi = ri.hi[g + 8 * r];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s = HL ? sc[t][i] + sc[t][2 + i] : sc[t][2 * r + i];
                s *= f;
                if (a.softcap_b > 0.f) s = a.softcap_b * tanhf(a.softcap_a * s);
                const int at = row0 + 8 * t + 2 * j + i;
                if (edge && (at < lo || at >= hi)) s = kNegInf;
                sc[t][2 * r + i] = s;
                move |= s > acc.m[r] + kLazy;
            }
    }
    if (__any_sync(0xffffffffu, move)) {
        float al[2] = {1.f, 1.f};
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float v = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            if (v > acc.m[r] + kLazy) {
                al[r] = acc.m[r] == kNegInf ? 0.f : ex2(acc.m[r] - v);
                acc.m[r] = v;
                acc.l[r] *= al[r];
            }
        }
        if (HL) al[1] = al[0];
#pragma unroll
        for (int n = 0; n < 4 * NB; ++n) {
            acc.o[n][0] *= al[0];
            acc.o[n][1] *= al[0];
            acc.o[n][2] *= al[1];
            acc.o[n][3] *= al[1];
        }
        if constexpr (HL && !F8) {
#pragma unroll
            for (int b = 0; b < NB; ++b) acc.mt[b] *= al[0];
        }
    }
    // ---- probabilities (a row without a reference yet has none but -inf scores)
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float s = sc[t][2 * r + i];
                const float p = s == kNegInf ? 0.f : ex2(s - acc.m[r] + kShift);
                acc.l[r] += p;
                sc[t][2 * r + i] = p;
            }
    // rows that no query sees may hold any bytes: their values are taken as 0
    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};           // half words of rows (2j, 2j+1), (2j+8, 2j+9)
    if (edge) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int at = row0 + 8 * t + 2 * j;
            const bool k0 = at >= ri.lo_min && at < ri.hi_max, k1 = at + 1 >= ri.lo_min && at + 1 < ri.hi_max;
            keep[t] = (k0 ? 0x0000ffffu : 0u) | (k1 ? 0xffff0000u : 0u);
        }
    }
    // ---- values
    uint4 pa;
    if constexpr (!HL) {
        pa.x = as_u32(__floats2half2_rn(sc[0][0], sc[0][1]));
        pa.y = as_u32(__floats2half2_rn(sc[0][2], sc[0][3]));
        pa.z = as_u32(__floats2half2_rn(sc[1][0], sc[1][1]));
        pa.w = as_u32(__floats2half2_rn(sc[1][2], sc[1][3]));
    } else if constexpr (F8) {
        const __half2 h0 = __floats2half2_rn(sc[0][0], sc[0][1]), h1 = __floats2half2_rn(sc[1][0], sc[1][1]);
        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
        pa.x = as_u32(h0);
        pa.z = as_u32(h1);
        pa.y = as_u32(__floats2half2_rn(sc[0][0] - f0.x, sc[0][1] - f0.y));
        pa.w = as_u32(__floats2half2_rn(sc[1][0] - f1.x, sc[1][1] - f1.y));
    }
    if constexpr (F8) {
        const uint32_t k0 = __byte_perm(keep[0], 0, 0x2020), k1 = __byte_perm(keep[1], 0, 0x2020);
        const uint32_t kb0 = k0, kb1 = k1;                   // bytes (row 2j, row 2j + 1) twice
        uint4 vv[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) vv[c] = *reinterpret_cast<const uint4*>(cell + 512 * NB + c * 512 + lane * 16);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int n0 = b, n1 = NB + b;
            const uint32_t x0 = (n0 & 1 ? vv[n0 / 2].z : vv[n0 / 2].x) & kb0, x1 = (n0 & 1 ? vv[n0 / 2].w : vv[n0 / 2].y) & kb0;
            const uint32_t y0 = (n1 & 1 ? vv[n1 / 2].z : vv[n1 / 2].x) & kb1, y1 = (n1 & 1 ? vv[n1 / 2].w : vv[n1 / 2].y) & kb1;
            mma_f16(acc.o[4 * b + 0], pa, f8_pair(x0), f8_pair(y0));
            mma_f16(acc.o[4 * b + 1], pa, f8_pair(x0 >> 16), f8_pair(y0 >> 16));
            mma_f16(acc.o[4 * b + 2], pa, f8_pair(x1), f8_pair(y1));
            mma_f16(acc.o[4 * b + 3], pa, f8_pair(x1 >> 16), f8_pair(y1 >> 16));
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
            uint4 dm = *reinterpret_cast<const uint4*>(cell + 864 * NB + (j * NB + b) * 16);
            dm.x &= keep[0]; dm.z &= keep[0];
            dm.y &= keep[1]; dm.w &= keep[1];
            const int n0 = b, n1 = NB + b;
            if constexpr (!HL) {
                auto tile = [&](auto R) {
                    constexpr int r = decltype(R)::value;
                    const __half2 c0 = __hsub2(as_h2(v_codes<r>(u[n0], nb[n0 / 4], n0 % 4, 0x64006400u)), as_h2(0x64006400u));
                    const __half2 c1 = __hsub2(as_h2(v_codes<r>(u[n1], nb[n1 / 4], n1 % 4, 0x64006400u)), as_h2(0x64006400u));
                    mma_f16(acc.o[4 * b + r], pa, as_u32(__hfma2(c0, as_h2(dm.x), as_h2(dm.z))),
                            as_u32(__hfma2(c1, as_h2(dm.y), as_h2(dm.w))));
                };
                tile(std::integral_constant<int, 0>{});
                tile(std::integral_constant<int, 1>{});
                tile(std::integral_constant<int, 2>{});
                tile(std::integral_constant<int, 3>{});
            } else {
                const float2 d0 = __half22float2(as_h2(dm.x)), d1 = __half22float2(as_h2(dm.y));
                const float2 m0 = __half22float2(as_h2(dm.z)), m1 = __half22float2(as_h2(dm.w));
                const float x0 = sc[0][0] * d0.x, x1 = sc[0][1] * d0.y, x2 = sc[1][0] * d1.x, x3 = sc[1][1] * d1.y;
                float t = acc.mt[b];
                t = fmaf(sc[0][0], fmaf(16.f, d0.x, m0.x), t);
                t = fmaf(sc[0][1], fmaf(16.f, d0.y, m0.y), t);
                t = fmaf(sc[1][0], fmaf(16.f, d1.x, m1.x), t);
                acc.mt[b] = fmaf(sc[1][1], fmaf(16.f, d1.y, m1.y), t);
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(x0, x1), h1 = __floats2bfloat162_rn(x2, x3);
                const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
                uint4 pd;
                pd.x = as_u32(h0);
                pd.z = as_u32(h1);
                pd.y = as_u32(__floats2bfloat162_rn(x0 - f0.x, x1 - f0.y));
                pd.w = as_u32(__floats2bfloat162_rn(x2 - f1.x, x3 - f1.y));
                auto tile = [&](auto R) {
                    constexpr int r = decltype(R)::value;
                    const __nv_bfloat162 mid = __floats2bfloat162_rn(144.f, 144.f);
                    uint32_t c0 = v_codes<r>(u[n0], nb[n0 / 4], n0 % 4, 0x43004300u);
                    uint32_t c1 = v_codes<r>(u[n1], nb[n1 / 4], n1 % 4, 0x43004300u);
                    c0 = as_u32(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&c0), mid));
                    c1 = as_u32(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&c1), mid));
                    mma_bf16(acc.o[4 * b + r], pd, c0, c1);
                };
                tile(std::integral_constant<int, 0>{});
                tile(std::integral_constant<int, 1>{});
                tile(std::integral_constant<int, 2>{});
                tile(std::integral_constant<int, 3>{});
            }
        }
    }
}

// Shared memory of the split kernel: query fragments, the join's sums, the
// plan, then a ring of `stages` cells per warp.
template <int NB, bool HL>
struct Smem {
    static constexpr int D = NB * 32;
    static constexpr size_t qs = (size_t)(D / 16) * 512;
    static constexpr size_t comb = (size_t)kCombine * (HL ? 8 : 16) * D * 4;
    __host__ __device__ static size_t ring(int E) { return (qs + comb + (size_t)(E + 1) * sizeof(PlanEntry) + 127) / 128 * 128; }
};

// Bounded wait for a stage; false once any wait of the CTA has run out.
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    if (dev::mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (dev::mbar_try_sleep(bar, parity, 20000u)) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > (1LL << 31)) {
            atomicExch(err, kErrWait);
            *abort_flag = 1;
            return false;
        }
    }
}

// A part of a CTA's range: key kk (KV head kh, slice sl) of entry e, cells [ca, cb)
struct Fragment {
    int e, kk, kh, sl, nsl, nq, c0, ca, cb, keys;
};
__device__ __forceinline__ Fragment fragment_at(const PlanEntry* plan, const SplitArgs& a, int QPI, long long x, long long x1) {
    Fragment f;
    f.e = find_entry(plan, a.E, x / a.g.Hkv);
    const PlanEntry pe = plan[f.e];
    const long long rel = x - pe.work * a.g.Hkv;
    f.kk = (int)(rel / pe.nc);
    f.ca = (int)(rel - (long long)f.kk * pe.nc);
    f.cb = (int)min((long long)pe.nc, f.ca + (x1 - x));
    f.nq = pe.pad;
    f.nsl = (pe.pad + QPI - 1) / QPI;
    f.kh = f.kk / f.nsl;
    f.sl = f.kk - f.kh * f.nsl;
    f.c0 = pe.c0;
    f.keys = pe.keys;
    return f;
}

// CTAs whose ranges meet a key: [first, last]; G ranges of W in all
__device__ __forceinline__ int cta_of(long long x, int G, long long W) { return (int)(((x + 1) * G - 1) / W); }

// The sums of one output row over records first + key .. last + key
template <int NB>
struct RowSum {
    float M, L, o[NB];
};
template <int NB>
__device__ __forceinline__ void fold_records(const SplitArgs& a, long long slot0, int n_rec, int rr, int lane, RowSum<NB>& r) {
    constexpr int D = NB * 32;
    for (int base = 0; base < n_rec; base += 32) {
        const int n = min(32, n_rec - base);
        float2 ml = make_float2(kNegInf, 0.f);
        if (lane < n) ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + ((slot0 + base + lane) * a.rec_rows + rr) * 2));
        float m = ml.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        m = fmaxf(m, r.M);
        if (m == kNegInf) continue;
        const float al = r.M == kNegInf ? 0.f : ex2(r.M - m);
        r.M = m;
        const float w = ml.x == kNegInf ? 0.f : ex2(ml.x - m);
        float l = ml.y * w;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
        r.L = r.L * al + l;
#pragma unroll
        for (int i = 0; i < NB; ++i) r.o[i] *= al;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float* src = a.part_o + ((slot0 + base + k) * a.rec_rows + rr) * D + lane;
#pragma unroll
            for (int i = 0; i < NB; ++i) r.o[i] = fmaf(wk, __ldcg(src + 32 * i), r.o[i]);
        }
    }
}

// Weight of a row's sums in its output, the sink taken in: out = o * weight
__device__ __forceinline__ float row_weight(const SplitArgs& a, int h, float M, float L) {
    if (M == kNegInf) return 0.f;
    if (a.sinks) {
        const float s = a.sinks[h] * 1.4426950408889634f;
        const float m = fmaxf(M, s);
        const float al = ex2(M - m);
        return al / (L * al + ex2(s - m));
    }
    return 1.0f / L;
}

template <int NB>
__device__ __forceinline__ void store_row(const SplitArgs& a, long long row, int h, int lane, const RowSum<NB>& r) {
    const float w = row_weight(a, h, r.M, r.L);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const long long at = row * (NB * 32) + 32 * i + lane;
        if (a.bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16(r.o[i] * w);
        else reinterpret_cast<float*>(a.out)[at] = r.o[i] * w;
    }
}

template <int NB, bool F8, bool HL>
__global__ void __launch_bounds__(warps_of<NB>() * 32, 1) split_kernel(const SplitArgs a, const int stages) {
    constexpr int D = NB * 32;
    constexpr int kWarps = warps_of<NB>(), kThreads = kWarps * 32;
    constexpr int QPI = HL ? 8 : 16;
    constexpr int NR = HL ? 1 : 2;
    constexpr int CELL = NB * (F8 ? 1024 : 928);
    using S = Smem<NB, HL>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint4* qs = reinterpret_cast<uint4*>(smem);
    float* comb = reinterpret_cast<float*>(smem + S::qs);
    PlanEntry* plan = reinterpret_cast<PlanEntry*>(smem + S::qs + S::comb);
    __shared__ RowInfo ri;
    __shared__ float s_m[kWarps][16], s_l[kWarps][16];
    __shared__ long long s_wsum[kWarps];
    __shared__ int s_ksum[kWarps];
    __shared__ int s_row0[kWarps][kMaxStages];        // first row of the cell in a stage, -1: none
    __shared__ __align__(8) uint64_t s_bar[kWarps][kMaxStages];
    __shared__ int s_abort, s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (lane < stages) dev::mbar_init(dev::smem_u32(&s_bar[warp][lane]), 1);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // ---- the plan: prefix sums of the entries' work
    {
        const int per = (a.E + kThreads - 1) / kThreads;
        long long w = 0;
        int k = 0;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < a.E) {
                const EntryWork ew = entry_work(a, e, blockIdx.x == 0);
                const int sl = (ew.nq + QPI - 1) / QPI;
                plan[e].nc = ew.nc;
                plan[e].c0 = ew.c0;
                plan[e].pad = ew.nq;
                plan[e].work = w;
                plan[e].keys = k;
                w += (long long)ew.nc * sl;
                k += sl;
            }
        }
        long long wi = w;
        int ki = k;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, wi, o);
            const int z = __shfl_up_sync(0xffffffffu, ki, o);
            if (lane >= o) {
                wi += y;
                ki += z;
            }
        }
        if (lane == 31) {
            s_wsum[warp] = wi;
            s_ksum[warp] = ki;
        }
        __syncthreads();
        long long wb = wi - w;
        int kb = ki - k;
        for (int i = 0; i < warp; ++i) {
            wb += s_wsum[i];
            kb += s_ksum[i];
        }
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < a.E) {
                plan[e].work += wb;
                plan[e].keys += kb;
            }
        }
        if (tid == kThreads - 1) {
            // groups that overlap could ask for more records than there are
            const bool fits = (long long)(kb + k) * a.g.Hkv <= a.max_keys;
            if (!fits) atomicExch(a.g.err, kErrCounter);
            plan[a.E].work = fits ? wb + w : 0;
            plan[a.E].keys = kb + k;
            plan[a.E].nc = plan[a.E].c0 = plan[a.E].pad = 0;
        }
        __syncthreads();
        if (!a.fuse && blockIdx.x == 0)
            for (int e = tid; e <= a.E; e += kThreads) a.plan[e] = plan[e];
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long W = plan[a.E].work * a.g.Hkv;
    const int G = (int)min((long long)a.G, W);
    if (a.fuse) {
        // entries without rows have no key: their outputs are zeros
        for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
            if (plan[e].nc != 0 && W != 0) continue;
            const long long at = (long long)e * (a.lists ? 1 : a.T) * a.Hq * D, n = (long long)(a.lists ? 1 : a.T) * a.Hq * D;
            for (long long i = tid; i < n; i += kThreads) {
                if (a.bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[at + i] = __float2bfloat16(0.f);
                else reinterpret_cast<float*>(a.out)[at + i] = 0.f;
            }
        }
    }
    if ((int)blockIdx.x >= G) return;
    const long long x0 = W * blockIdx.x / G, x1 = W * (blockIdx.x + 1) / G;
    const int cpp = a.g.cells_per_page();
    const uint32_t ring = dev::smem_u32(smem) + (uint32_t)S::ring(a.E) + (uint32_t)(warp * stages * CELL);
    const uint8_t* ring_p = smem + S::ring(a.E) + (size_t)warp * stages * CELL;
    const uint32_t bar0 = dev::smem_u32(&s_bar[warp][0]);

    // ---- the producer side of this warp's ring: its cells (every kWarps-th of
    // each fragment) in order, `stages` ahead of their use.  Lanes look up the
    // pages of 32 cells at once.
    long long px = x0;                                  // first cell after the producer's fragment
    int pc = 0, pcb = 0, pslot = -1, ppage = -1, pidx = 32;
    const int* ptable = nullptr;
    const int* plist = nullptr;
    int pkh = 0, pc0 = 0, phi = 0;
    auto produce = [&](int st) {
        if (pc >= pcb) {
            // the next fragment in which this warp has a cell
            for (;;) {
                if (px >= x1) return;
                const Fragment f = fragment_at(plan, a, QPI, px, x1);
                px += f.cb - f.ca;
                pc = f.ca + warp;
                if (pc >= f.cb) continue;
                pcb = f.cb;
                pc0 = f.c0;
                pkh = f.kh;
                int seq = f.e;
                if (a.lists) seq = f.e / a.T;
                else if (f.e >= a.n_seq) seq = a.group_start[f.e - a.n_seq];
                ptable = a.tables + (long long)seq * a.g.max_pages;
                plist = a.lists ? a.lists + ((long long)f.e * a.g.Hkv + f.kh) * a.keep : nullptr;
                phi = a.lists ? a.lens[seq] - a.T + (f.e - seq * a.T) + 1 : 0x7fffffff;
                pidx = 32;
                break;
            }
        }
        if (pidx == 32) {
            pidx = 0;
            const int c = pc + lane * kWarps;
            pslot = ppage = -1;
            if (c < pcb) {
                if (plist) {
                    pslot = plist[c / cpp];
                    if (pslot >= a.g.max_pages) {
                        atomicExch(a.g.err, kErrCounter);
                        pslot = -1;
                    }
                    if (pslot >= 0 && pslot * a.g.page_rows + (c % cpp) * 16 >= phi) pslot = -1;
                } else {
                    pslot = (pc0 + c) / cpp;
                }
                if (pslot >= 0) ppage = ptable[pslot];
                if (pslot >= 0 && (ppage < 0 || ppage >= a.g.n_pages)) {
                    atomicExch(a.g.err, kErrCounter);
                    ppage = -1;
                }
            }
        }
        const int page = __shfl_sync(0xffffffffu, ppage, pidx), slot = __shfl_sync(0xffffffffu, pslot, pidx);
        if (lane == 0) {
            const uint32_t bar = bar0 + 8u * st;
            const int in = (plist ? pc : pc0 + pc) % cpp;
            if (page >= 0) {
                s_row0[warp][st] = slot * a.g.page_rows + in * 16;
                dev::mbar_expect_tx(bar, CELL);
                dev::bulk_g2s(ring + (uint32_t)(st * CELL), a.g.pool + page * a.g.page_bytes + (long long)(pkh * cpp + in) * CELL, CELL, bar);
            } else {
                s_row0[warp][st] = -1;
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
            }
        }
        ++pidx;
        pc += kWarps;
    };
    for (int st = 0; st < stages; ++st) produce(st);

    int st = 0;
    uint32_t phase = 0;
    long long x = x0;
    while (x < x1) {
        const Fragment f = fragment_at(plan, a, QPI, x, x1);
        const long long xa = plan[f.e].work * a.g.Hkv + (long long)f.kk * plan[f.e].nc, xb = xa + plan[f.e].nc;
        x += f.cb - f.ca;

        // ---- its queries, as A fragments in shared memory
        __syncthreads();
        for (int r = warp; r < QPI; r += kWarps) {
            const int qi = f.sl * QPI + r;
            Query q{0, 0, 0, 0, -1};
            float v[NB];
            float am = 0.f;
            const bool valid = qi < f.nq;
            if (valid) q = query_of(a, f.e, f.kh, qi);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                v[b] = valid ? load_q(a.q, (((long long)q.seq * a.T + q.t) * a.Hq + q.h) * D + 32 * b + lane, a.bf16) : 0.f;
                am = fmaxf(am, fabsf(v[b]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            // scaled by a power of two to a largest element in [512, 1024)
            const int ex = am > 0.f ? min(max((int)(__float_as_uint(am) >> 23) - 127 - 9, -117), 118) : 0;
            const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (lane == 0) {
                ri.fac[r] = a.qscale * __uint_as_float((uint32_t)(127 + ex) << 23);
                ri.lo[r] = q.lo;
                ri.hi[r] = q.hi;
            }
            const int wi = lane & 7, j = lane >> 3;
            const int reg = ((wi & 3) >> 1) * 2, half = wi & 1;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float y = v[b] * up;
                const __half hi = __float2half_rn(y);
                __half* dst = reinterpret_cast<__half*>(qs + (2 * b + (wi >> 2)) * 32 + 4 * (r & 7) + j);
                if (HL) {
                    dst[2 * reg + half] = hi;
                    dst[2 * (reg + 1) + half] = __float2half_rn(y - __half2float(hi));
                } else {
                    dst[2 * (reg + (r >> 3)) + half] = hi;
                }
            }
        }
        __syncthreads();
        if (warp == 0) {
            const bool v = lane < QPI && f.sl * QPI + lane < f.nq;
            int lo_max = v ? ri.lo[lane] : 0, hi_min = v ? ri.hi[lane] : 0x7fffffff;
            int lo_min = v ? ri.lo[lane] : 0x7fffffff, hi_max = v ? ri.hi[lane] : 0;
            if (v && ri.hi[lane] <= ri.lo[lane]) lo_min = 0x7fffffff, hi_max = 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, o));
                hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, o));
                lo_min = min(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
                hi_max = max(hi_max, __shfl_xor_sync(0xffffffffu, hi_max, o));
            }
            if (lane == 0) {
                ri.lo_max = lo_max;
                ri.hi_min = hi_min;
                ri.lo_min = lo_min;
                ri.hi_max = hi_max;
            }
        }
        __syncthreads();

        Acc<NB, F8, HL> acc;
#pragma unroll
        for (int n = 0; n < 4 * NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc.o[n][i] = 0.f;
        acc.m[0] = acc.m[1] = kNegInf;
        acc.l[0] = acc.l[1] = 0.f;
#pragma unroll
        for (int b = 0; b < (HL && !F8 ? NB : 1); ++b) acc.mt[b] = 0.f;

        // ---- its cells, warp by warp
        for (int c = f.ca + warp; c < f.cb; c += kWarps) {
            const bool there = wait_stage(bar0 + 8u * st, phase, &s_abort, a.g.err);
            const int row0 = s_row0[warp][st];
            if (there && row0 >= 0 && row0 < ri.hi_max)
                take_cell<NB, F8, HL>(a, ring_p + st * CELL, row0, qs, ri, lane, acc);
            __syncwarp();
            if (there) produce(st);
            if (++st == stages) {
                st = 0;
                phase ^= 1u;
            }
        }

        // ---- join the warps: common reference, then sums passed down four warps at a time
        const int g = lane >> 2, j = lane & 3;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], 1);
            acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], 2);
            if (j == 0) {
                s_m[warp][g + 8 * r] = acc.m[r];
                s_l[warp][g + 8 * r] = acc.l[r];
            }
        }
        if constexpr (HL) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float t = 0.f;
                if constexpr (!F8) {
                    t = acc.mt[b];
                    t += __shfl_xor_sync(0xffffffffu, t, 1);
                    t += __shfl_xor_sync(0xffffffffu, t, 2);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc.o[4 * b + r][0] += acc.o[4 * b + r][2] + t;
                    acc.o[4 * b + r][1] += acc.o[4 * b + r][3] + t;
                }
            }
        }
        __syncthreads();
        float M[2], L[2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            M[r] = kNegInf;
            L[r] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M[r] = fmaxf(M[r], s_m[w][g + 8 * r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (s_m[w][g + 8 * r] != kNegInf) L[r] += s_l[w][g + 8 * r] * ex2(s_m[w][g + 8 * r] - M[r]);
            const float fa = acc.m[r] == kNegInf ? 0.f : ex2(acc.m[r] - M[r]);
#pragma unroll
            for (int n = 0; n < 4 * NB; ++n) {
                acc.o[n][2 * r] *= fa;
                acc.o[n][2 * r + 1] *= fa;
            }
        }
        auto pass = [&](int lo, int n) {               // warps [lo + n, lo + 2n) add their sums to [lo, lo + n)
            float2* buf = reinterpret_cast<float2*>(comb) + (size_t)(warp & (n - 1)) * (4 * NB * NR * 32);
            if (warp >= lo + n && warp < lo + 2 * n) {
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        buf[(i * NR + r) * 32 + lane] = make_float2(acc.o[i][2 * r], acc.o[i][2 * r + 1]);
            }
            __syncthreads();
            if (warp >= lo && warp < lo + n) {
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i)
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        const float2 y = buf[(i * NR + r) * 32 + lane];
                        acc.o[i][2 * r] += y.x;
                        acc.o[i][2 * r + 1] += y.y;
                    }
            }
            __syncthreads();
        };
        for (int lo = kWarps - 2 * kCombine; lo >= 0; lo -= kCombine) pass(lo, kCombine);
        for (int n = kCombine / 2; n >= 1; n >>= 1) pass(0, n);

        const int cta0 = cta_of(xa, G, W), n_rec = cta_of(xb - 1, G, W) - cta0 + 1;
        const long long key = (long long)f.keys * a.g.Hkv + f.kk;
        const int rows = min(QPI, f.nq - f.sl * QPI);
        if (warp == 0) {
            const bool whole = a.fuse && n_rec == 1;
            const long long slot = blockIdx.x + key;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int row = g + 8 * r;
                if (row >= rows) continue;
                if (whole) {
                    const Query q = query_of(a, f.e, f.kh, f.sl * QPI + row);
                    const float w = row_weight(a, q.h, M[r] == kNegInf ? kNegInf : M[r] - kShift, L[r]);
                    const long long at = (((long long)q.seq * a.T + q.t) * a.Hq + q.h) * D + 8 * j;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = acc.o[4 * b + (i & 3)][2 * r + (i >> 2)] * w;
                        if (a.bf16) {
                            uint32_t w4[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w4[i] = as_u32(__floats2bfloat162_rn(y[2 * i], y[2 * i + 1]));
                            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at + 32 * b) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        } else {
                            float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at + 32 * b);
                            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    continue;
                }
                float* dst = a.part_o + (slot * a.rec_rows + row) * D + 8 * j;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    *reinterpret_cast<float4*>(dst + 32 * b) = make_float4(acc.o[4 * b][2 * r], acc.o[4 * b + 1][2 * r], acc.o[4 * b + 2][2 * r], acc.o[4 * b + 3][2 * r]);
                    *reinterpret_cast<float4*>(dst + 32 * b + 4) = make_float4(acc.o[4 * b][2 * r + 1], acc.o[4 * b + 1][2 * r + 1], acc.o[4 * b + 2][2 * r + 1], acc.o[4 * b + 3][2 * r + 1]);
                }
                if (j == 0)
                    *reinterpret_cast<float2*>(a.part_ml + (slot * a.rec_rows + row) * 2) =
                        make_float2(M[r] == kNegInf ? kNegInf : M[r] - kShift, L[r]);
            }
            if (a.fuse && n_rec > 1) {
                // the CTA that completes a key's records joins them; the others go on
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const bool last = atomicAdd(a.arrived + key, 1) == n_rec - 1;
                    if (last) a.arrived[key] = 0;
                    s_last = last;
                    __threadfence();
                }
            }
        }
        if (a.fuse && n_rec > 1) {
            __syncthreads();
            if (s_last) {
                for (int rr = warp; rr < rows; rr += kWarps) {
                    RowSum<NB> r;
                    r.M = kNegInf;
                    r.L = 0.f;
#pragma unroll
                    for (int i = 0; i < NB; ++i) r.o[i] = 0.f;
                    fold_records<NB>(a, cta0 + key, n_rec, rr, lane, r);
                    const Query q = query_of(a, f.e, f.kh, f.sl * QPI + rr);
                    store_row<NB>(a, ((long long)q.seq * a.T + q.t) * a.Hq + q.h, q.h, lane, r);
                }
            }
        }
    }
    if (s_abort) {                                     // a wait ran out: let copies in flight land before the CTA ends
        const long long t0 = clock64();
        while (clock64() - t0 < (1LL << 30)) __nanosleep(1000);
    }
}

// ------------------------------------------------------------ merge kernel

// One warp per output row (sequence, t, head) of a shared decode: the records
// of its own rows' key and of its group's prefix, and the sink.
template <int NB>
__global__ void __launch_bounds__(256) merge_kernel(const SplitArgs a, int QPI) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= (long long)a.n_seq * a.T * a.Hq) return;
    const int h = (int)(row % a.Hq), st = (int)(row / a.Hq);
    const int seq = st / a.T, t = st - seq * a.T;
    const int kh = h / a.hpk, hr = h - kh * a.hpk;
    const long long W = a.plan[a.E].work * a.g.Hkv;
    const int G = (int)min((long long)a.G, W);
    RowSum<NB> r;
    r.M = kNegInf;
    r.L = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) r.o[i] = 0.f;
    auto fold = [&](int e, int qi) {
        const PlanEntry pe = a.plan[e];
        if (pe.nc == 0 || W == 0) return;
        const int nsl = (pe.pad + QPI - 1) / QPI;
        const int kk = kh * nsl + qi / QPI;
        const long long xa = pe.work * a.g.Hkv + (long long)kk * pe.nc;
        const int c0 = cta_of(xa, G, W), c1 = cta_of(xa + pe.nc - 1, G, W);
        fold_records<NB>(a, (long long)pe.keys * a.g.Hkv + kk + c0, c1 - c0 + 1, qi % QPI, lane, r);
    };
    fold(seq, t * a.hpk + hr);
    const int grp = group_of(a, seq);
    if (grp >= 0) {
        int gs, ge;
        members(a, grp, gs, ge);
        if (seq >= gs && seq < ge) fold(a.n_seq + grp, ((seq - gs) * a.T + t) * a.hpk + hr);
    }
    store_row<NB>(a, row, h, lane, r);
}

template <int NB, bool F8, bool HL>
cudaError_t launch_split_t(const SplitArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(split_kernel<NB, F8, HL>, done, true);
    if (e != cudaSuccess) return e;
    using S = Smem<NB, HL>;
    constexpr size_t cells = (size_t)warps_of<NB>() * NB * (F8 ? 1024 : 928);
    // the ring takes what the plan leaves of 220 KB (2 to 8 stages)
    const int stages = (int)std::min<size_t>(kMaxStages, (220 * 1024 - S::ring(a.E)) / cells);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.G);
    cfg.blockDim = dim3(warps_of<NB>() * 32);
    cfg.dynamicSmemBytes = S::ring(a.E) + stages * cells;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, split_kernel<NB, F8, HL>, a, stages);
}

template <int NB>
cudaError_t launch_split_nb(const SplitArgs& a, cudaStream_t s) {
    if (a.g.fp8) return a.bf16 ? launch_split_t<NB, true, false>(a, s) : launch_split_t<NB, true, true>(a, s);
    return a.bf16 ? launch_split_t<NB, false, false>(a, s) : launch_split_t<NB, false, true>(a, s);
}

}  // namespace

int split_queries(const SplitArgs& a) { return a.bf16 ? 16 : 8; }

cudaError_t launch_split(const SplitArgs& a, cudaStream_t s) {
    switch (a.g.NB()) {
        case 2: return launch_split_nb<2>(a, s);
        case 4: return launch_split_nb<4>(a, s);
        default: return launch_split_nb<8>(a, s);
    }
}

cudaError_t launch_merge(const SplitArgs& a, cudaStream_t s) {
    const long long rows = (long long)a.n_seq * a.T * a.Hq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int qpi = split_queries(a);
    switch (a.g.NB()) {
        case 2: return cudaLaunchKernelEx(&cfg, merge_kernel<2>, a, qpi);
        case 4: return cudaLaunchKernelEx(&cfg, merge_kernel<4>, a, qpi);
        default: return cudaLaunchKernelEx(&cfg, merge_kernel<8>, a, qpi);
    }
}

}  // namespace paged
}  // namespace kvq
