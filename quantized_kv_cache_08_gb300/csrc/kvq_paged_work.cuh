// Device helpers shared by the paged decode kernels: conversions of codes, work
// entries, queries and the rows they see, bounded waits.
#pragma once

#include "kvq_device.cuh"
#include "kvq_paged.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace kvq {
namespace paged {

using dev::kLazy;
using dev::kNegInf;
constexpr float kShift = 6.0f;         // p is held as 2^6 p: fp16 keeps 2^-20 of the largest in full
constexpr int kMaxStages = 8;
constexpr float kNone = -3.402823466e38f;   // reference of a query that has seen no row: no score lies below it
constexpr float kInf = __builtin_huge_valf();
constexpr uint32_t kInfBits = 0x7f800000u;

// A score's factor inside f32's normal numbers: 0 x -inf (a masked row) and 0 x inf
// (a key of zeros) would be NaN.  Scores that the bounds move are far below any
// rounding, or beyond f32 unless they are 0.
__device__ __forceinline__ float factor(float f) { return fminf(fmaxf(f, 1.17549435e-38f), 3.402823466e38f); }

// Sum of a fragment's weights as its record has it, and whether the query saw a row.
// A query that is not finite goes through the products as zeros (`bad`) and a score
// that overflows leaves the reference at infinity: both make the sum NaN, which every
// join keeps, so that the output is NaN however the work was cut.
__device__ __forceinline__ bool settle(float& l, float m, bool bad) {
    const bool seen = l > 0.f || m == kInf;
    if (seen && (bad || m == kInf)) l = __uint_as_float(0x7fffffffu);
    return seen;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// two E4M3 bytes as a half pair, exact
__device__ __forceinline__ uint32_t f8_pair(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// (x & mask) | y in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t y) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "r"(mask), "r"(y));
    return d;
}
// A constant that the compiler keeps in a register (an instruction takes one
// immediate, so a mask and a magic number as constants would make two of one)
__device__ __forceinline__ uint32_t held(uint32_t c) {
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(c));
    return r;
}
// The 5-bit codes of element R of two rows, in the low bits of each half word, on
// top of `magic`; the element 3 nibbles are at bit 4 n4 of nib's half words
template <int R>
__device__ __forceinline__ uint32_t v_codes(uint32_t unit, uint32_t nib, int n4, uint32_t magic) {
    if constexpr (R == 0) return and_or(unit, 0x001f001fu, magic);
    else if constexpr (R == 1) return and_or(unit >> 5, 0x001f001fu, magic);
    else if constexpr (R == 2) return and_or(unit >> 10, 0x001f001fu, magic);
    else return and_or(nib >> (4 * n4), 0x000f000fu, and_or(unit >> 11, 0x00100010u, magic));
}

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

// code bytes (biased by 128) sel of w under the exponent of 1024, minus 1152: exact
__device__ __forceinline__ uint32_t k_pair(uint32_t w, uint32_t sel, uint32_t exps) {
    return as_u32(__hsub2(as_h2(__byte_perm(w, exps, sel)), as_h2(0x64806480u)));
}
__device__ __forceinline__ float load_q(const void* q, long long idx, int bf16) {
    if (bf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[idx]);
    return reinterpret_cast<const float*>(q)[idx];
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

// A group whose queries per KV head are more than one slice of the split kernel
// goes to the tile kernel: the split kernel reads the rows again for each slice.
// Whole calls with the groups in either, 8 KV heads of 128, 16 rows of each
// sequence's own (tile / split / a dense decode, us):
//   queries   2048 rows         8192 rows
//        9    40 / 27 / 23      54 / 34 / 40
//       64    43 / 30 / 28      56 / 43 / 59
//      128    44 / 38 / 41      56 / 59 / 101
//      256    48 / 49 / 63      63 / 91 / 186
// The tile kernel pays from about 128 queries over 8192 rows on; in smaller groups
// its start and end, some 25 us, are more than the reading that it saves.
__device__ __forceinline__ bool tile_group(const SplitArgs& a, int nq) { return a.tiles && nq > a.tile; }

struct EntryWork {
    int nc, c0, nq;
    int rows, lo;                  // as in PlanEntry
};

__device__ __forceinline__ EntryWork entry_work(const SplitArgs& a, int e, bool report) {
    EntryWork w{0, 0, 0, 0, 0};
    int lo = 0, hi = 0;
    if (a.lists) {
        const int seq = e / a.T, t = e - seq * a.T;
        const int len = a.lens[seq];
        if (!len_ok(a, len)) {
            if (report) atomicExch(a.g.err, kErrCounter);
            return w;
        }
        w.nq = a.hpk;
        w.rows = len;
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
        w.rows = len;
        if (grp >= 0) w.lo = prefix_rows(a, grp);
        lo = max(lo, w.lo);
    } else {
        const int grp = e - a.n_seq;
        int gs, ge;
        members(a, grp, gs, ge);
        if (report && (a.group_start[grp + 1] < a.group_start[grp] || a.group_start[grp] < 0 ||
                       a.group_start[grp + 1] > a.n_seq || !len_ok(a, a.prefix_len[grp])))
            atomicExch(a.g.err, kErrCounter);
        w.nq = (ge - gs) * a.hpk * a.T;
        if (tile_group(a, w.nq)) return EntryWork{0, 0, 0, 0, 0};
        hi = prefix_rows(a, grp);
        lo = 0;
        w.rows = hi;
        w.lo = gs;
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
__device__ __forceinline__ Query query_of(const SplitArgs& a, const PlanEntry& pe, int e, int g, int qi) {
    Query q;
    int within = qi, len = pe.rows;
    if (a.lists) {
        q.seq = e / a.T;
        q.t = e - q.seq * a.T;
    } else {
        q.seq = e;
        if (e >= a.n_seq) {
            const int Qh = a.hpk * a.T, m = qi / Qh;
            q.seq = pe.lo + m;
            within = qi - m * Qh;
            len = a.lens[q.seq];
            if (!len_ok(a, len)) len = 0;
        }
        q.t = within / a.hpk;
        within -= q.t * a.hpk;
    }
    q.h = g * a.hpk + within;
    q.hi = len - a.T + q.t + 1;
    q.lo = a.window > 0 ? max(0, q.hi - a.window) : 0;
    if (e >= a.n_seq && !a.lists) q.hi = min(q.hi, pe.rows);
    else q.lo = max(q.lo, pe.lo);
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

// Bounded wait; false once any wait of the CTA has run out.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
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

}  // namespace paged
}  // namespace kvq
