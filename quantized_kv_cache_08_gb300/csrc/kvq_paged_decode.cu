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
// a key has); f32 queries keep f32 accuracy with tiles of 8: rows 0..7 of the S
// tile carry the high part of the queries and rows 8..15 the low part, two fp16
// numbers (22 bits of a query scaled to its largest element), and P d goes in as
// two bf16 numbers (16 bits, any range) against the exact codes u - 16, with
// sum p (m + 16 d) kept in f32 beside it.
//
// Why tensor cores for one token: the products cost the same for 1 or 8 queries,
// so the work that grows with the bytes is the unpacking alone, where the
// multiply-add form needs as many instructions again for each 4 queries.
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
constexpr int kMaxGroups = 4;          // groups of warps in a CTA

// Query tiles: 8 or 16 bf16 queries, or 8 of f32 in two parts
enum Tile { kT8 = 0, kT16 = 1, kF32 = 2 };

// Warps of a CTA (one CTA an SM): as many as the accumulators leave registers for
template <int NB, int TILE>
constexpr int warps_of() { return NB == 8 ? 8 : NB == 4 && TILE == kT16 ? 12 : 16; }
template <int TILE>
constexpr int queries_of() { return TILE == kT16 ? 16 : 8; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c = a b, without a sum to start from
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
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

template <int NB, bool F8, int TILE>
struct Acc {
    static constexpr int NQ = TILE == kT16 ? 2 : 1;       // groups of 8 queries
    // O^T tile 2b + rp of a group: rows g / g + 8 are elements 32b + 4g + 2rp and
    // + 1, columns 2j, 2j + 1 queries: [0] (el, 2j) [1] (el, 2j+1) [2] (el+1, 2j) ..
    float o[NQ][2 * NB][4];
    float m[NQ], l[NQ];                                   // query g (+ 8): reference, sum of p
    float mt[TILE == kF32 && !F8 ? NB : 1];               // sum p (m + 16 d) of query g
};

struct RowInfo {
    float fac[16];
    int lo[16], hi[16];
    int lo_min, lo_max, hi_min, hi_max;
};

// Per-lane facts of a fragment's queries g (+ 8)
template <int NQ>
struct LaneRows {
    float fac[NQ];
    int lo[NQ], hi[NQ];
};

constexpr float kNone = -1e30f;        // reference of a query that has seen no row: any score passes it

// Values of rows that no query sees, in the staged cell: zeroed, for they may be any bytes
template <int NB, bool F8>
__device__ __forceinline__ void clear_rows(uint8_t* cell, int row0, const RowInfo& ri, int lane) {
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
                                          const RowInfo& ri, const LaneRows<Acc<NB, F8, TILE>::NQ>& lr, int lane,
                                          Acc<NB, F8, TILE>& acc) {
    constexpr bool HL = TILE == kF32;
    constexpr int NQ = Acc<NB, F8, TILE>::NQ;
    const int j = lane & 3;
    const bool edge = row0 < ri.lo_max || row0 + 16 > ri.hi_min;
    if (edge) clear_rows<NB, F8>(cell, row0, ri, lane);
    // ---- scores
    float sc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[t][i] = 0.f;
    auto q_frag = [&](int step) {
        if constexpr (TILE == kT8) {
            const uint2 x = *reinterpret_cast<const uint2*>(qs + (step * 32 + lane) * 8);
            return make_uint4(x.x, 0u, x.y, 0u);
        } else {
            return *reinterpret_cast<const uint4*>(qs + (step * 32 + lane) * 16);
        }
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
            const uint4 a0 = q_frag(2 * b), a1 = q_frag(2 * b + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t w0 = e ? kk[t].z : kk[t].x, w1 = e ? kk[t].w : kk[t].y;
                if constexpr (F8) {
                    mma_f16(sc[t], a0, f8_pair(w0), f8_pair(w0 >> 16));
                    mma_f16(sc[t], a1, f8_pair(w1), f8_pair(w1 >> 16));
                } else {
                    float c[4];
                    mma_f16_new(c, a0, k_pair(w0, 0x4140u), k_pair(w0, 0x4342u));
                    mma_f16(c, a1, k_pair(w1, 0x4140u), k_pair(w1, 0x4342u));
                    const float2 d = __half22float2(as_h2(e ? (t ? ks.w : ks.z) : (t ? ks.y : ks.x)));
                    if constexpr (HL) {
                        c[0] += c[2];
                        c[1] += c[3];
                    }
                    sc[t][0] = fmaf(c[0], d.x, sc[t][0]);
                    sc[t][1] = fmaf(c[1], d.y, sc[t][1]);
                    if constexpr (TILE == kT16) {
                        sc[t][2] = fmaf(c[2], d.x, sc[t][2]);
                        sc[t][3] = fmaf(c[3], d.y, sc[t][3]);
                    }
                }
            }
        }
    }
    if constexpr (HL && F8) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            sc[t][0] += sc[t][2];
            sc[t][1] += sc[t][3];
        }
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
                for (int b = 0; b < NB; ++b) acc.mt[b] *= al;
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
    uint32_t pl[2];                                       // low parts (E4M3 rows, f32 queries)
#pragma unroll
    for (int r = 0; r < NQ; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t) pb[r][t] = as_u32(__floats2half2_rn(sc[t][2 * r], sc[t][2 * r + 1]));
    if constexpr (HL && F8) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float2 f = __half22float2(as_h2(pb[0][t]));
            pl[t] = as_u32(__floats2half2_rn(sc[t][0] - f.x, sc[t][1] - f.y));
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
                if constexpr (HL) mma_f16(acc.o[0][2 * b + rp], va, pl[0], pl[1]);
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
                    const __half2 c = __hsub2(as_h2(v_codes<r>(u[n], nb[n / 4], n % 4, 0x64006400u)), as_h2(0x64006400u));
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
                const float x0 = sc[0][0] * d0.x, x1 = sc[0][1] * d0.y, x2 = sc[1][0] * d1.x, x3 = sc[1][1] * d1.y;
                float t = acc.mt[b];
                t = fmaf(sc[0][0], fmaf(16.f, d0.x, m0.x), t);
                t = fmaf(sc[0][1], fmaf(16.f, d0.y, m0.y), t);
                t = fmaf(sc[1][0], fmaf(16.f, d1.x, m1.x), t);
                acc.mt[b] = fmaf(sc[1][1], fmaf(16.f, d1.y, m1.y), t);
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(x0, x1), h1 = __floats2bfloat162_rn(x2, x3);
                const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
                const uint32_t ph0 = as_u32(h0), ph1 = as_u32(h1);
                const uint32_t pl0 = as_u32(__floats2bfloat162_rn(x0 - f0.x, x1 - f0.y));
                const uint32_t pl1 = as_u32(__floats2bfloat162_rn(x2 - f1.x, x3 - f1.y));
                auto code = [&](auto R, int n) {
                    constexpr int r = decltype(R)::value;
                    uint32_t c = v_codes<r>(u[n], nb[n / 4], n % 4, 0x43004300u);
                    return as_u32(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&c), __floats2bfloat162_rn(144.f, 144.f)));
                };
                const std::integral_constant<int, 0> r0{};
                const std::integral_constant<int, 1> r1{};
                const std::integral_constant<int, 2> r2{};
                const std::integral_constant<int, 3> r3{};
                const uint4 v0 = make_uint4(code(r0, n0), code(r1, n0), code(r0, n1), code(r1, n1));
                mma_bf16(acc.o[0][2 * b], v0, ph0, ph1);
                mma_bf16(acc.o[0][2 * b], v0, pl0, pl1);
                const uint4 v1 = make_uint4(code(r2, n0), code(r3, n0), code(r2, n1), code(r3, n1));
                mma_bf16(acc.o[0][2 * b + 1], v1, ph0, ph1);
                mma_bf16(acc.o[0][2 * b + 1], v1, pl0, pl1);
            }
        }
    }
    // the stage's next copy comes by another proxy than clear_rows' writes
    if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared memory of the split kernel: query fragments of each group, the joins'
// sums, the plan, then a ring of `stages` cells per warp.
template <int NB, int TILE>
struct Smem {
    static constexpr int D = NB * 32;
    static constexpr size_t qs = (size_t)(D / 16) * (TILE == kT8 ? 256 : 512);
    static constexpr size_t comb = (size_t)warps_of<NB, TILE>() / 2 * queries_of<TILE>() * D * 4;
    __host__ __device__ static size_t ring(int E) { return (kMaxGroups * qs + comb + (size_t)(E + 1) * sizeof(PlanEntry) + 127) / 128 * 128; }
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

// A part of a range: key kk (KV head kh, slice sl) of entry e, cells [ca, cb)
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

// Ranges that W cells are cut into: one for each group of warps, and a cell
// for each of its warps at least, so that a short context is joined from few
// records
__device__ __forceinline__ int ranges(const SplitArgs& a, long long W) {
    return (int)min((long long)a.G * a.groups, (W + a.gw - 1) / a.gw);
}

// The range that holds cell x; G ranges of W cells in all
__device__ __forceinline__ int range_of(long long x, int G, long long W) { return (int)(((x + 1) * G - 1) / W); }

// The sums of one output row over its key's records; a lane holds elements
// 2 lane, + 1 (NB 2) or 4 lane .. + 3 of each 128
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
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float* src = a.part_o + ((slot0 + base + k) * a.rec_rows + rr) * D;
            if constexpr (NB == 2) {
                const float2 y = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                r.o[0] = fmaf(wk, y.x, r.o[0]);
                r.o[1] = fmaf(wk, y.y, r.o[1]);
            } else {
#pragma unroll
                for (int i = 0; i < NB; i += 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(src) + 8 * i + lane);
                    r.o[i] = fmaf(wk, y.x, r.o[i]);
                    r.o[i + 1] = fmaf(wk, y.y, r.o[i + 1]);
                    r.o[i + 2] = fmaf(wk, y.z, r.o[i + 2]);
                    r.o[i + 3] = fmaf(wk, y.w, r.o[i + 3]);
                }
            }
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
    for (int i = 0; i < NB; i += 2) {
        const long long at = row * (NB * 32) + (NB == 2 ? 2 * lane : 32 * (i & ~3) + 4 * lane + (i & 2));
        const float x = r.o[i] * w, y = r.o[i + 1] * w;
        if (a.bf16) *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + at) = as_u32(__floats2bfloat162_rn(x, y));
        else *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = make_float2(x, y);
    }
}

template <int NB, bool F8, int TILE>
__global__ void __launch_bounds__(warps_of<NB, TILE>() * 32, 1) split_kernel(const SplitArgs a, const int stages) {
    constexpr int D = NB * 32;
    constexpr int kWarps = warps_of<NB, TILE>(), kThreads = kWarps * 32;
    constexpr bool HL = TILE == kF32;
    constexpr int QPI = queries_of<TILE>(), NQ = QPI / 8;
    constexpr int CELL = NB * (F8 ? 1024 : 928);
    using S = Smem<NB, TILE>;
    extern __shared__ __align__(128) uint8_t smem[];
    PlanEntry* plan = reinterpret_cast<PlanEntry*>(smem + kMaxGroups * S::qs + S::comb);
    __shared__ RowInfo s_ri[kMaxGroups];
    __shared__ float s_m[kWarps][16], s_l[kWarps][16];
    __shared__ long long s_wsum[kWarps];
    __shared__ int s_ksum[kWarps];
    __shared__ int s_row0[kWarps][kMaxStages];        // first row of the cell in a stage, -1: none
    __shared__ __align__(8) uint64_t s_bar[kWarps][kMaxStages];
    __shared__ int s_abort, s_last[kMaxGroups];
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
    const int G = ranges(a, W);
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
    // ---- the CTA's groups of gw warps work on ranges of their own: while one
    // group joins and changes keys (some 5 us of latencies) the others compute
    const int gw = a.gw, group = warp / gw, gwarp = warp - group * gw;
    const int range = group * gridDim.x + blockIdx.x;
    if (range >= G) return;
    const long long x0 = W * range / G, x1 = W * (range + 1) / G;
    uint8_t* qs = smem + group * S::qs;
    float* comb = reinterpret_cast<float*>(smem + kMaxGroups * S::qs) + (size_t)group * (gw / 2) * QPI * D;
    RowInfo& ri = s_ri[group];
    auto sync_group = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gw * 32) : "memory"); };
    const int cpp = a.g.cells_per_page(), cps = a.g.page_shift - 4;       // cells a page, a power of two
    const uint32_t ring = dev::smem_u32(smem) + (uint32_t)S::ring(a.E) + (uint32_t)(warp * stages * CELL);
    uint8_t* ring_p = smem + S::ring(a.E) + (size_t)warp * stages * CELL;
    const uint32_t bar0 = dev::smem_u32(&s_bar[warp][0]);

    // ---- the producer side of this warp's ring: its cells (every gw-th of
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
                pc = f.ca + gwarp;
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
            const int c = pc + lane * gw;
            pslot = ppage = -1;
            if (c < pcb) {
                if (plist) {
                    pslot = plist[c >> cps];
                    if (pslot >= a.g.max_pages) {
                        atomicExch(a.g.err, kErrCounter);
                        pslot = -1;
                    }
                    if (pslot >= 0 && pslot * a.g.page_rows + (c & (cpp - 1)) * 16 >= phi) pslot = -1;
                } else {
                    pslot = (pc0 + c) >> cps;
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
            const int in = (plist ? pc : pc0 + pc) & (cpp - 1);
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
        pc += gw;
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
        sync_group();
        for (int r = gwarp; r < QPI; r += gw) {
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
                const int at = (2 * b + (wi >> 2)) * 32 + 4 * (r & 7) + j;
                __half* dst = reinterpret_cast<__half*>(qs + at * (TILE == kT8 ? 8 : 16));
                if (TILE == kT8) {
                    dst[reg + half] = hi;
                } else if (HL) {
                    dst[2 * reg + half] = hi;
                    dst[2 * (reg + 1) + half] = __float2half_rn(y - __half2float(hi));
                } else {
                    dst[2 * (reg + (r >> 3)) + half] = hi;
                }
            }
        }
        sync_group();
        if (gwarp == 0) {
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
        sync_group();

        const int g = lane >> 2, j = lane & 3;
        Acc<NB, F8, TILE> acc;
        LaneRows<NQ> lr;
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
        for (int b = 0; b < (HL && !F8 ? NB : 1); ++b) acc.mt[b] = 0.f;

        // ---- its cells, warp by warp
        for (int c = f.ca + gwarp; c < f.cb; c += gw) {
            const bool there = wait_stage(bar0 + 8u * st, phase, &s_abort, a.g.err);
            const int row0 = s_row0[warp][st];
            if (there && row0 >= 0 && row0 < ri.hi_max)
                take_cell<NB, F8, TILE>(a, ring_p + st * CELL, row0, qs, ri, lr, lane, acc);
            __syncwarp();
            if (there) produce(st);
            if (++st == stages) {
                st = 0;
                phase ^= 1u;
            }
        }

        // ---- join the group's warps: common reference, then sums passed down
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
            for (int b = 0; b < NB; ++b) {
                float t = acc.mt[b];
                t += __shfl_xor_sync(0xffffffffu, t, 1);
                t += __shfl_xor_sync(0xffffffffu, t, 2);
                const float t0 = __shfl_sync(0xffffffffu, t, 8 * j), t1 = __shfl_sync(0xffffffffu, t, 8 * j + 4);
#pragma unroll
                for (int rp = 0; rp < 2; ++rp) {
                    acc.o[0][2 * b + rp][0] += t0;
                    acc.o[0][2 * b + rp][1] += t1;
                    acc.o[0][2 * b + rp][2] += t0;
                    acc.o[0][2 * b + rp][3] += t1;
                }
            }
        }
        sync_group();
        float M[NQ][2], L[NQ][2];                          // of queries 2j, 2j + 1 (+ 8)
#pragma unroll
        for (int r = 0; r < NQ; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 2 * j + i + 8 * r;
                float m = kNone, l = 0.f;
                const int w0 = warp - gwarp;
#pragma unroll 4
                for (int w = w0; w < w0 + gw; ++w) m = fmaxf(m, s_m[w][row]);
#pragma unroll 4
                for (int w = w0; w < w0 + gw; ++w) l = fmaf(s_l[w][row], ex2(s_m[w][row] - m), l);
                const float fa = ex2(s_m[warp][row] - m);
#pragma unroll
                for (int n = 0; n < 2 * NB; ++n) {
                    acc.o[r][n][i] *= fa;
                    acc.o[r][n][2 + i] *= fa;
                }
                M[r][i] = l > 0.f ? m - kShift : kNegInf;
                L[r][i] = l;
            }
        auto pass = [&](int lo, int n) {               // warps [lo + n, lo + 2n) add their sums to [lo, lo + n)
            float4* buf = reinterpret_cast<float4*>(comb) + (size_t)(gwarp & (n - 1)) * (2 * NB * NQ * 32);
            if (gwarp >= lo + n && gwarp < lo + 2 * n) {
#pragma unroll
                for (int r = 0; r < NQ; ++r)
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i)
                        buf[(r * 2 * NB + i) * 32 + lane] = make_float4(acc.o[r][i][0], acc.o[r][i][1], acc.o[r][i][2], acc.o[r][i][3]);
            }
            sync_group();
            if (gwarp >= lo && gwarp < lo + n) {
#pragma unroll
                for (int r = 0; r < NQ; ++r)
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) {
                        const float4 y = buf[(r * 2 * NB + i) * 32 + lane];
                        acc.o[r][i][0] += y.x;
                        acc.o[r][i][1] += y.y;
                        acc.o[r][i][2] += y.z;
                        acc.o[r][i][3] += y.w;
                    }
            }
            sync_group();
        };
        const int n0 = gw & (gw - 1) ? 4 : gw / 2;         // 12 warps: 4 onto 4 onto 4
        for (int lo = gw - 2 * n0; lo >= 0; lo -= n0) pass(lo, n0);
        for (int n = n0 / 2; n >= 1; n >>= 1) pass(0, n);

        const int rec0 = range_of(xa, G, W), n_rec = range_of(xb - 1, G, W) - rec0 + 1;
        const long long key = (long long)f.keys * a.g.Hkv + f.kk;
        const int rows = min(QPI, f.nq - f.sl * QPI);
        if (gwarp == 0) {
            const bool whole = a.fuse && n_rec == 1;
            const long long slot = range + key;
#pragma unroll
            for (int r = 0; r < NQ; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = 2 * j + i + 8 * r;
                    if (row >= rows) continue;
                    if (whole) {
                        const Query q = query_of(a, f.e, f.kh, f.sl * QPI + row);
                        const float w = row_weight(a, q.h, M[r][i], L[r][i]);
                        const long long at = (((long long)q.seq * a.T + q.t) * a.Hq + q.h) * D + 4 * g;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const float y0 = acc.o[r][2 * b][i] * w, y1 = acc.o[r][2 * b][2 + i] * w;
                            const float y2 = acc.o[r][2 * b + 1][i] * w, y3 = acc.o[r][2 * b + 1][2 + i] * w;
                            if (a.bf16)
                                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at + 32 * b) =
                                    make_uint2(as_u32(__floats2bfloat162_rn(y0, y1)), as_u32(__floats2bfloat162_rn(y2, y3)));
                            else
                                *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at + 32 * b) = make_float4(y0, y1, y2, y3);
                        }
                        continue;
                    }
                    float* dst = a.part_o + (slot * a.rec_rows + row) * D + 4 * g;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        *reinterpret_cast<float4*>(dst + 32 * b) = make_float4(acc.o[r][2 * b][i], acc.o[r][2 * b][2 + i], acc.o[r][2 * b + 1][i], acc.o[r][2 * b + 1][2 + i]);
                    if (g == 0)
                        *reinterpret_cast<float2*>(a.part_ml + (slot * a.rec_rows + row) * 2) = make_float2(M[r][i], L[r][i]);
                }
            if (a.fuse && n_rec > 1) {
                // the group that completes a key's records joins them; the others go on
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const bool last = atomicAdd(a.arrived + key, 1) == n_rec - 1;
                    if (last) a.arrived[key] = 0;
                    s_last[group] = last;
                    __threadfence();
                }
            }
        }
        if (a.fuse && n_rec > 1) {
            sync_group();
            if (s_last[group]) {
                for (int rr = gwarp; rr < rows; rr += gw) {
                    RowSum<NB> r;
                    r.M = kNegInf;
                    r.L = 0.f;
#pragma unroll
                    for (int i = 0; i < NB; ++i) r.o[i] = 0.f;
                    fold_records<NB>(a, rec0 + key, n_rec, rr, lane, r);
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
    const int G = ranges(a, W);
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
        const int c0 = range_of(xa, G, W), c1 = range_of(xa + pe.nc - 1, G, W);
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

template <int NB, bool F8, int TILE>
cudaError_t launch_split_t(const SplitArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(split_kernel<NB, F8, TILE>, done, true);
    if (e != cudaSuccess) return e;
    using S = Smem<NB, TILE>;
    constexpr size_t cells = (size_t)warps_of<NB, TILE>() * NB * (F8 ? 1024 : 928);
    // the ring takes what the plan leaves of 220 KB
    const int stages = (int)std::min<size_t>(kMaxStages, (220 * 1024 - S::ring(a.E)) / cells);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.G);
    cfg.blockDim = dim3(warps_of<NB, TILE>() * 32);
    cfg.dynamicSmemBytes = S::ring(a.E) + stages * cells;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, split_kernel<NB, F8, TILE>, a, stages);
}

template <int NB, bool F8>
cudaError_t launch_split_f(const SplitArgs& a, cudaStream_t s) {
    if (!a.bf16) return launch_split_t<NB, F8, kF32>(a, s);
    return a.tile == 8 ? launch_split_t<NB, F8, kT8>(a, s) : launch_split_t<NB, F8, kT16>(a, s);
}

template <int NB>
cudaError_t launch_split_nb(const SplitArgs& a, cudaStream_t s) {
    return a.g.fp8 ? launch_split_f<NB, true>(a, s) : launch_split_f<NB, false>(a, s);
}

}  // namespace

int split_tile(bool bf16, int most_queries) { return bf16 && most_queries > 8 ? 16 : 8; }

int split_warps(int NB, int tile) {
    if (tile == 16) return NB == 2 ? warps_of<2, kT16>() : NB == 4 ? warps_of<4, kT16>() : warps_of<8, kT16>();
    return NB == 2 ? warps_of<2, kT8>() : NB == 4 ? warps_of<4, kT8>() : warps_of<8, kT8>();
}
static_assert(warps_of<2, kT8>() == warps_of<2, kF32>() && warps_of<4, kT8>() == warps_of<4, kF32>() &&
              warps_of<8, kT8>() == warps_of<8, kF32>(), "tiles of 8 queries share a CTA size");

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
    switch (a.g.NB()) {
        case 2: return cudaLaunchKernelEx(&cfg, merge_kernel<2>, a, a.tile);
        case 4: return cudaLaunchKernelEx(&cfg, merge_kernel<4>, a, a.tile);
        default: return cudaLaunchKernelEx(&cfg, merge_kernel<8>, a, a.tile);
    }
}

}  // namespace paged
}  // namespace kvq
