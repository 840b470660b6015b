// Paged cache: append with the position rotation applied on the way, rows read
// back as values, and the key bounds of pages.
//
// Append.  A group of D / 8 lanes takes one head row of one token, 8 elements a
// lane; four lanes hold a 32-element block.  Queries and keys are rotated in
// registers (the partner half comes by shuffles, so queries may be rotated in
// place), keys become q8_0 codes, values q5_1 codes, or both E4M3 bytes, and go
// to their places in the page's cell.  The angles of a CTA's tokens are worked
// out once into shared memory and serve all heads.  8k rows of 32 query and 8 KV
// heads of 128: 52 us where the bytes take 27; 38.7 M instructions (the exact
// rounding of every code) keep two thirds of the issue slots busy, the rest waits
// for loads, shuffles and the angles' barriers; 64 rows 4.8 us.
//
// Angles.  With f in turns per position held as f_hi + f_lo (48 bits), p f_hi
// splits exactly into a rounded product and its error (fma), the whole turns
// drop out exactly, and the rest is added: the angle is good to 2^-24 of a turn
// at any position below 2^24, where p f in one fp32 product would be off by
// p 2^-24 radians.  Positions are a row's index in its sequence, or given for each
// row on up to four axes, of which each pair of elements has one; those angles are worked out
// further (put_angle_at; 8k rows 55.3 us in all, by index 51.0).  bf16 instances without
// bounds spill 76 to 104 bytes a thread at their 64 registers.
#include "kvq_paged.cuh"
#include "kvq_quant.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCellThreads = 128, kCellWarps = kCellThreads / 32;
constexpr int kTT = 4;                 // tokens of a CTA when there are many (2: 64 us, 8: 57 us where 4 takes 56)

// Eight elements as they lie in memory, then as floats
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ void fetch8(const void* base, long long idx, Raw8<BF16>& r) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) + idx * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.w[i] = p[i];
}
template <bool BF16>
__device__ __forceinline__ void floats8(const Raw8<BF16>& r, float (&x)[8]) {
    if constexpr (BF16) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
}

__device__ __forceinline__ void store8(void* base, long long idx, int bf16, const float (&x)[8]) {
    if (bf16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + idx) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + idx);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// fp16 of the exact quotient (num + err) / den, to nearest even in one rounding
// (den 127 or 31; num >= 0, err what num as a float leaves out).  The fp32
// quotient decides unless it lies within a few of its own steps of a midpoint
// between two halves (low 13 bits near 0x1000): there num is compared with
// midpoint x den, which is exact in fp32 (12 + 7 bits), as is the difference.
// Subnormal halves are left to fp64.
__device__ __forceinline__ unsigned short half_quotient(float num, float err, float den) {
    const float q = __fdiv_rn(num, den);
    if (q < 6.2e-5f) return __half_as_ushort(__double2half(((double)num + (double)err) / (double)den));
    const uint32_t bits = __float_as_uint(q), low = bits & 0x1fffu;
    if (low >= 0x0ff8u && low <= 0x1008u) {
        const uint32_t down = bits & ~0x1fffu;
        const float r = (num - __uint_as_float(down | 0x1000u) * den) + err;
        const bool up = r > 0.f || (r == 0.f && ((down >> 13) & 1u));
        return __half_as_ushort(__float2half_rn(__uint_as_float(up ? down + 0x2000u : down)));
    }
    return __half_as_ushort(__float2half_rn(q));
}

// Stored rows are finite whatever comes in: a row that one query does not see
// meets it with weight 0 in the same matrix product as the queries that see it,
// and 0 x inf would reach its output; and a key's scores are numbers for every
// query.  A q8_0 element stays within +-kKeyEnd, the largest that a scale of fp16
// holds, a NaN is zero.  A q5_1 block's ends stay within +-65280, so
// that 31 d + m with d rounded up (by 2^-12, here up to 64 in all) stays below
// fp16's 65504; an infinite element takes the code at that end, a NaN the lowest, a
// block of NaN is zeros.  An E4M3 NaN is zero.
__device__ __forceinline__ void bound_block(float& least, float& most) {
    if (!(least <= most)) least = most = 0.f;
    least = fminf(fmaxf(least, -65280.f), 65280.f);
    most = fminf(fmaxf(most, -65280.f), 65280.f);
}
__device__ __forceinline__ float number(float x) { return x == x ? x : 0.f; }
constexpr float kKeyEnd = 65504.f * 127.f;

// The rotation table of a token holds (cos, sin) of pair p at place
// (p % 8) (n / 8) + p / 8 (4 for interleaved pairs) of n: the lanes of a load,
// which take neighbouring groups of pairs, read neighbouring words.
// (cos, sin) of pair pr at position pos into a token's table of `half` pairs
__device__ __forceinline__ void put_angle(float2* cs_of, float2 f, int pos, int pr, int half, int interleaved) {
    const float p = (float)max(pos, 0);
    const float t = p * f.x;
    const float e = fmaf(p, f.x, -t);
    const float turn = (t - rintf(t)) + fmaf(p, f.y, e);
    float sn, cs;
    sincospif(2.f * turn, &sn, &cs);
    const int grp = interleaved ? 4 : 8;
    cs_of[(pr % grp) * (half / grp) + pr / grp] = make_float2(cs, sn);
}

// A row's given positions (asked for before its place is known: the two chains of loads overlap)
__device__ __forceinline__ void load_positions(const AppendArgs& a, int row, int (&at)[kMaxAxes]) {
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) at[x] = x < a.n_axes ? a.positions[(long long)row * a.n_axes + x] : 0;
}
// All -1, and the error word set, where one is out of range
__device__ __forceinline__ void check_positions(const AppendArgs& a, int (&at)[kMaxAxes]) {
    bool ok = true;
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) ok = ok && at[x] >= 0 && at[x] < kMaxPosition;
    if (ok) return;
    atomicExch(a.g.err, kErrCounter);
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) at[x] = -1;
}

// The row scores of a row just placed start at 0: KV heads h, h + step ..
__device__ __forceinline__ void clear_scores(const AppendArgs& a, const Place& p, int h, int step) {
    const int in = p.pos & (a.g.page_rows - 1);
    const long long page = (p.cell - (long long)(in >> 4) * a.g.cell_bytes) / a.g.page_bytes;
    for (; h < a.g.Hkv; h += step) a.row_scores[(page * a.g.Hkv + h) * a.g.page_rows + in] = 0.f;
}

// The same for a given position, to nearly the last bit of f32: E4M3 codes lie so far
// apart that whatever an angle is off moves some of them over a border.  The rounding
// errors of products and sums are carried along, so that the turn is off by no more
// than its frequency leaves out; from the nearest quarter the angle z = zh + zl is
// within pi / 4, where in
//   sin z = zh + (zl + zh^3 S(zh^2)), cos z = 1 - zh^2 / 2 + (zh^4 C(zh^2) - zh zl)
// (S and C by their Taylor series) the terms in brackets are small: 0.6 of a last bit.
// Some 50 operations a pair.
__device__ __forceinline__ void put_angle_at(float2* cs_of, float2 f, int pos, int pr, int half, int interleaved) {
    const float p = (float)max(pos, 0);
    const float t = __fmul_rn(p, f.x), e = __fmaf_rn(p, f.x, -t);               // p f.x = t + e
    const float m = __fmul_rn(p, f.y), ml = __fmaf_rn(p, f.y, -m);              // p f.y = m + ml
    float s = __fadd_rn(e, m), b = __fadd_rn(s, -e);
    const float sl = __fadd_rn(__fadd_rn(e, -__fadd_rn(s, -b)), __fadd_rn(m, -b));      // e + m = s + sl
    s = __fadd_rn(s, -rintf(s));
    const float a = __fadd_rn(t, -rintf(t));
    float h = __fadd_rn(a, s);
    b = __fadd_rn(h, -a);
    const float hl = __fadd_rn(__fadd_rn(a, -__fadd_rn(h, -b)), __fadd_rn(s, -b));      // a + s = h + hl
    const float lo = __fadd_rn(hl, __fadd_rn(sl, ml));
    const float q = rintf(4.f * h);                                             // quarters
    const int k = (int)q;
    h = __fmaf_rn(q, -0.25f, h);                                                // (exact)
    const float two_pi = 6.28318548f, rest = -1.74845553e-7f;                   // 2 pi as a sum of two floats
    const float zh = __fmul_rn(h, two_pi);
    const float zl = __fadd_rn(__fmaf_rn(h, two_pi, -zh), __fmaf_rn(h, rest, __fmul_rn(lo, two_pi)));
    const float z2 = __fmul_rn(zh, zh);
    float S = -2.50521084e-8f;                                                  // -1 / 11!, 1 / 9! ..
    S = __fmaf_rn(S, z2, 2.75573192e-6f);
    S = __fmaf_rn(S, z2, -1.98412698e-4f);
    S = __fmaf_rn(S, z2, 8.33333333e-3f);
    S = __fmaf_rn(S, z2, -1.66666667e-1f);
    const float sn = __fadd_rn(zh, __fmaf_rn(__fmul_rn(z2, zh), S, zl));
    float C = 2.08767570e-9f;                                                   // 1 / 12!, -1 / 10! ..
    C = __fmaf_rn(C, z2, -2.75573192e-7f);
    C = __fmaf_rn(C, z2, 2.48015873e-5f);
    C = __fmaf_rn(C, z2, -1.38888889e-3f);
    C = __fmaf_rn(C, z2, 4.16666667e-2f);
    const float hz = __fmul_rn(0.5f, z2), w = __fadd_rn(1.f, -hz);
    const float left = __fadd_rn(__fadd_rn(__fadd_rn(1.f, -w), -hz), __fmul_rn(-0.5f, __fmaf_rn(zh, zh, -z2)));      // what w leaves of 1 - zh^2 / 2
    const float cs = __fadd_rn(w, __fadd_rn(left, __fmaf_rn(__fmul_rn(z2, z2), C, -__fmul_rn(zh, zl))));
    float c = k & 1 ? sn : cs, n = k & 1 ? cs : sn;
    if ((k + 1) & 2) c = -c;
    if (k & 2) n = -n;
    const int grp = interleaved ? 4 : 8;
    cs_of[(pr % grp) * (half / grp) + pr / grp] = make_float2(c, n);
}

// Rotate elements e0 .. e0 + 7 (x) below rot of a head row; y: those that the half-split rotation pairs them with
__device__ __forceinline__ void turn8(float (&x)[8], const float (&y)[8], int e0, int rot, int interleaved, const float2* cs) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = cs[i * (rot / 8) + e0 / 8];
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = p * a.x - q * a.y;
            x[2 * i + 1] = p * a.y + q * a.x;
        }
        return;
    }
    const int half = rot / 2;
    const bool second = e0 >= half;
    const float2* c = cs + (second ? e0 - half : e0) / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 a = c[i * (half / 8)];
        x[i] = second ? y[i] * a.y + x[i] * a.x : x[i] * a.x - y[i] * a.y;
    }
}

// Rotate the 8 elements e0.. of a head row; every lane of the warp calls this
// (shuffles).
__device__ __forceinline__ void rotate8(float (&x)[8], int e0, int rot, int interleaved, const float2* cs, int lane) {
    if (rot == 0) return;
    if (interleaved) {
        if (e0 < rot) turn8(x, x, e0, rot, 1, cs);
        return;
    }
    const int half = rot / 2, from = e0 < rot ? lane + (e0 >= half ? -half / 8 : half / 8) : lane;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
    if (e0 < rot) turn8(x, y, e0, rot, 0, cs);
}

// Codes of 8 elements by q8_0's or q5_1's rule: round-half-away(t) for t = x / d
// or (x - m) / d, clamped.  Adding 1.5 * 2^23 leaves the nearest integer in the
// low bits of the sum; t itself is off by less than 2e-5.  Where it lies within
// 1e-4 of k + 1/2 the exact rule decides: 2 |x| >= (2k + 1) d, both sides exact
// in fp32 (d has 11 bits, the odd number 8), or the same of x - m with the part
// that its float leaves out.  Subnormal scales are left to the fp64 rule.
template <bool V>
__device__ __forceinline__ void codes8(const float (&x)[8], float m, float d, int (&code)[8]) {
    constexpr float kMagic = 12582912.f;
    const float inv = d > 0.f ? 1.0f / d : 0.f;
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float t = (V ? x[i] - m : x[i]) * inv;
        if (V) t = fminf(fmaxf(t, -0.25f), 31.25f);
        const float y = t + kMagic;
        near |= fabsf(t - (y - kMagic)) > 0.4999f;
        const int c = __float_as_int(y) - __float_as_int(kMagic);
        code[i] = V ? min(max(c, 0), 31) : c;
    }
    if (d < 6.2e-5f) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float xi = x[0];
#pragma unroll
            for (int k = 1; k < 8; ++k)
                if (k == i) xi = x[k];
            const int c = d > 0.f ? (V ? q5_code(xi, m, d, inv) : q8_code(xi, d, inv)) : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k == i) code[k] = c;
        }
    } else if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = V ? x[i] - m : x[i];
            const float z = s - x[i];
            const float e = V ? (x[i] - (s - z)) - (m + z) : 0.f;        // x - m = s + e
            const float t = fabsf(s * inv);
            const float k = floorf(t);
            if (fabsf(t - k - 0.5f) < 1e-4f && !(V && (s < 0.f || k > 30.f))) {
                const float r = (2.f * fabsf(s) - (2.f * k + 1.f) * d) + (s < 0.f ? -2.f : 2.f) * e;
                const int n = (int)k + (r >= 0.f ? 1 : 0);
                code[i] = s < 0.f ? -n : n;
            }
        }
    }
}

// Bounds of the 8 elements of lane c of a block as codes: rounded outward in
// steps of ds = max |k| / 127.
__device__ __forceinline__ void store_bounds(int8_t* codes, float* scales, long long at, int c, float ds, const float* mn, const float* mx) {
    uint32_t lo[2] = {0u, 0u}, hi[2] = {0u, 0u};
    if (ds > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float l = fminf(fmaxf(floorf(__fdiv_rn(mn[i], ds)), -127.f), 127.f);
            const float u = fminf(fmaxf(ceilf(__fdiv_rn(mx[i], ds)), -127.f), 127.f);
            lo[i >> 2] |= ((uint32_t)(int)l & 255u) << (8 * (i & 3));
            hi[i >> 2] |= ((uint32_t)(int)u & 255u) << (8 * (i & 3));
        }
    }
    int8_t* dst = codes + at * 64 + 8 * c;
    *reinterpret_cast<uint2*>(dst) = make_uint2(lo[0], lo[1]);
    *reinterpret_cast<uint2*>(dst + 32) = make_uint2(hi[0], hi[1]);
    if (c == 0) scales[at] = ds;
}

// Least and greatest of the 8 elements that lane (b, c) holds, over the first
// `rows` rows of a page's head: 16 rows' codes and scales in flight at a time.
template <int NB>
__device__ __forceinline__ void fold_rows(const uint8_t* cell, long long step, int fp8, int rows, int b, int c, float (&mn)[8], float (&mx)[8]) {
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 16, cell += step) {
        uint2 w[16], d[4];
#pragma unroll
        for (int t = 0; t < 16; ++t)
            if (r0 + t < rows) w[t] = *reinterpret_cast<const uint2*>(cell + (b >> 1) * 1024 + t * 64 + c * 16 + (b & 1) * 8);
        if (!fp8)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = *reinterpret_cast<const uint2*>(cell + 512 * NB + (j * NB + b) * 8);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            if (r0 + t >= rows) continue;
            const int j = (t & 7) >> 1;
            const uint32_t dw = (t >> 3) ? d[j].y : d[j].x;
            const float s = fp8 ? 1.f : __half2float(__ushort_as_half((unsigned short)(dw >> (16 * (t & 1)))));
            const uint32_t w2[2] = {w[t].x, w[t].y};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = (w2[i >> 2] >> (8 * (i & 3))) & 255u;
                const float x = fp8 ? __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)u, __NV_E4M3))) : (float)((int)u - 128) * s;
                mn[i] = fminf(mn[i], x);
                mx[i] = fmaxf(mx[i], x);
            }
        }
    }
}

// Query units u0, u0 + du .. of a token (64 / LR heads each) rotated into q_out by
// one warp.  A lane's two pieces: partners of the half-split rotation, else side
// by side.
template <int LR, bool BF16>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, long long row, const float2* cs, int u0, int du, int lane) {
    constexpr int D = LR * 8, QPW = 64 / LR, QL = LR / 2;
    const int half = a.rope_dim / 2, uq = a.q ? (a.Hq + QPW - 1) / QPW : 0;
    const int ql = lane % QL, split = a.interleaved ? 0 : a.rope_dim / 16;
    const int qa = 8 * (ql < split ? ql : split + 2 * (ql - split) + (a.interleaved ? 0 : split));
    const int qb = ql < split ? qa + half : qa + 8;
    constexpr int U = BF16 ? 2 : 1;                // units in flight
    for (int u = u0; u < uq; u += U * du) {
        Raw8<BF16> rx[U], ry[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = (u + k * du) * QPW + lane / QL;
            if (h < a.Hq) {
                fetch8(a.q, row * a.q_stride + h * D + qa, rx[k]);
                fetch8(a.q, row * a.q_stride + h * D + qb, ry[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = (u + k * du) * QPW + lane / QL;
            if (h >= a.Hq) continue;           // (no shuffles on this path)
            float x[8], y[8];
            floats8(rx[k], x);
            floats8(ry[k], y);
            if (a.interleaved) {
                rotate8(x, qa, a.rope_dim, 1, cs, lane);
                rotate8(y, qb, a.rope_dim, 1, cs, lane);
            } else if (ql < split) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 c = cs[i * (half / 8) + ql];
                    const float p = x[i], q = y[i];
                    x[i] = p * c.x - q * c.y;
                    y[i] = p * c.y + q * c.x;
                }
            }
            store8(a.q_out, (row * a.Hq + h) * D + qa, BF16, x);
            store8(a.q_out, (row * a.Hq + h) * D + qb, BF16, y);
        }
    }
}

// One append CTA: tokens [TT blockIdx.x, + TT), row units blockIdx.y, + gridDim.y..
// A unit is a warp's rows of one kind of one token: 64 / LR query heads (a lane
// holds 8 elements and the 8 that they are rotated with), or 32 / LR key or
// value heads (8 elements a lane, four lanes a block).
// MORE: positions are given, or scores kept (apart, for the branches alone cost an
// append of 8k rows 1 us and a step 0.2).
template <int LR, bool BF16, bool BOUNDS, bool MORE>
__global__ void __launch_bounds__(kThreads, BOUNDS ? 2 : BF16 ? 4 : 3) append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ Freqs fq, int TT) {
    extern __shared__ float2 s_cs[];               // [TT][rope_dim / 2]
    __shared__ Place s_place[kTT];
    __shared__ int s_at[MORE ? kTT : 1][kMaxAxes]; // given positions
    constexpr int D = LR * 8, NB = D / 32, JPW = 32 / LR, QPW = 64 / LR;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row0 = blockIdx.x * TT;
    const int half = a.rope_dim / 2;
    wait_for_earlier();
    let_next_start();
    if (warp == 0) {
        const int row = row0 + lane;
        [[maybe_unused]] int at[kMaxAxes] = {};
        if (MORE && a.positions && lane < TT && row < a.r.rows) load_positions(a, row, at);
        const int i = entry_of_rows<kTT>(a.r, row0, lane);
        Place p{-1, -1, 0, 0, 0};
        if (lane < TT && row < a.r.rows) p = place_in(a.g, a.r, row, i, true);
        if (MORE && a.positions && p.pos >= 0) {
            check_positions(a, at);
            if (at[0] < 0) p = Place{-1, -2, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < kMaxAxes; ++x) s_at[lane][x] = at[x];
        }
        if (lane < TT) s_place[lane] = p;
    }
    __syncthreads();
    // (an indexed read of the frequencies takes a step for each lane: one a thread)
    for (int pr = tid % (kThreads / TT); pr < half; pr += kThreads / TT) {
        const int tt = tid / (kThreads / TT);
        if (MORE && a.positions) {
            if (s_place[tt].pos >= 0) put_angle_at(s_cs + tt * half, fq.f[pr], s_at[tt][fq.axis[pr]], pr, half, a.interleaved);
        } else {
            put_angle(s_cs + tt * half, fq.f[pr], s_place[tt].pos, pr, half, a.interleaved);
        }
    }
    __syncthreads();
    // a warp's token, and its share of the token's units
    const int wpt = kWarps / TT, tt = warp / wpt;
    const int u0 = blockIdx.y * wpt + warp - tt * wpt, du = gridDim.y * wpt;
    const Place pl = s_place[tt];
    if (pl.pos < 0) return;
    if (MORE && a.row_scores && blockIdx.y == 0 && pl.cell >= 0) clear_scores(a, pl, (warp - tt * wpt) * 32 + lane, wpt * 32);
    const float2* cs = s_cs + tt * half;
    const long long row = row0 + tt;
    const int uq = a.q ? (a.Hq + QPW - 1) / QPW : 0, uk = (a.g.Hkv + JPW - 1) / JPW;
    rotate_queries<LR, BF16>(a, row, cs, u0, du, lane);
    // the first unit of keys and values that is this warp's
    int u = u0 >= uq ? u0 : u0 + (uq - u0 + du - 1) / du * du;
    // ---- keys and values
    const int li = lane % LR, e0 = 8 * li;
    const int t = pl.t, b = li >> 2, c = li & 3;
    const int j = (t & 7) >> 1, s = t & 1, hh = t >> 3;
    const int n = hh * NB + b, i4 = 2 * hh + s;
    Raw8<BF16> next{};                             // of the unit after the one in work
    auto fetch = [&](int u) {
        const bool is_v = u >= uq + uk;
        const int h = (is_v ? u - uk - uq : u - uq) * JPW + lane / LR;
        if (u < uq + 2 * uk && h < a.g.Hkv && pl.cell >= 0)
            fetch8(is_v ? a.v : a.k, row * (is_v ? a.v_stride : a.k_stride) + h * D + e0, next);
    };
    fetch(u);
    for (; u < uq + 2 * uk; u += du) {
        const bool is_v = u >= uq + uk;
        const int h = (is_v ? u - uk - uq : u - uq) * JPW + lane / LR;
        const bool on = h < a.g.Hkv && pl.cell >= 0;
        float x[8], mn[8], mx[8];
        uint8_t* cell = a.g.pool + pl.cell + (long long)h * a.g.cells_per_page() * a.g.cell_bytes;
        const int in = pl.pos & (a.g.page_rows - 1);       // row of the page
        if constexpr (BOUNDS) {                            // the page's earlier rows, while this one's elements are on their way
            if (!is_v) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    mn[i] = __builtin_huge_valf();
                    mx[i] = -__builtin_huge_valf();
                }
                fold_rows<NB>(cell - (long long)(in >> 4) * a.g.cell_bytes, a.g.cell_bytes, a.g.fp8, on ? in : 0, b, c, mn, mx);
            }
        }
        floats8(next, x);
        fetch(u + du);
        if (!is_v) {
            rotate8(x, e0, a.rope_dim, a.interleaved, cs, lane);
            uint32_t w2[2] = {0u, 0u};
            float kd = 0.f;
            if (a.g.fp8) {
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    w2[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(number(x[i]), number(x[i + 1])), __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
            } else {
                // the largest |element|, by its bits: NaN lies above infinity
                auto largest = [&]() {
                    uint32_t m = 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    return __uint_as_float(m);
                };
                float m = largest();
                if (__any_sync(0xffffffffu, !(m <= kKeyEnd))) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(number(x[i]), -kKeyEnd), kKeyEnd);
                    m = largest();
                }
                const unsigned short db = half_quotient(m, 0.f, 127.f);
                int code[8];
                kd = __half2float(__ushort_as_half(db));
                codes8<false>(x, 0.f, kd, code);
#pragma unroll
                for (int i = 0; i < 8; i += 4)
                    w2[i >> 2] = __byte_perm(__byte_perm(code[i], code[i + 1], 0x0040), __byte_perm(code[i + 2], code[i + 3], 0x0040), 0x5410) ^ 0x80808080u;
                if (on && c == 0)
                    *reinterpret_cast<unsigned short*>(cell + 512 * NB + (j * NB + b) * 8 + i4 * 2) = db;
            }
            if (on) *reinterpret_cast<uint2*>(cell + (b >> 1) * 1024 + t * 64 + c * 16 + (b & 1) * 8) = make_uint2(w2[0], w2[1]);
            if constexpr (BOUNDS) {                // this row's values as stored, from registers
                float am = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u = (w2[i >> 2] >> (8 * (i & 3))) & 255u;
                    const float y = a.g.fp8 ? __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)u, __NV_E4M3)))
                                            : (float)((int)u - 128) * kd;
                    mn[i] = fminf(mn[i], y);
                    mx[i] = fmaxf(mx[i], y);
                    am = fmaxf(am, fmaxf(fabsf(mn[i]), fabsf(mx[i])));
                }
                am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
                const long long page = (pl.cell - (long long)(in >> 4) * a.g.cell_bytes) / a.g.page_bytes;
                if (on) store_bounds(a.codes, a.scales, (page * a.g.Hkv + h) * NB + b, c, __fmul_rn(am, 1.0f / 127.0f), mn, mx);
            }
            continue;
        }
        if (a.g.fp8) {
            uint8_t* p = cell + 512 * NB + (n >> 1) * 512 + (n & 1) * 8 + s;
            if (on) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    p[(4 * (2 * c + (i >> 2)) + j) * 16 + (i & 3) * 2] =
                        __nv_cvt_float_to_fp8(number(x[i]), __NV_SATFINITE, __NV_E4M3);
            }
            continue;
        }
        float least = x[0], most = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            least = fminf(least, x[i]);
            most = fmaxf(most, x[i]);
        }
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, 2));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        bound_block(least, most);
        const float range = most - least, back = range - most;
        const unsigned short db = half_quotient(range, (most - (range - back)) - (least + back), 31.f);
        const unsigned short mb = __half_as_ushort(__float2half_rn(least));
        int code[8];
        codes8<true>(x, __half2float(__ushort_as_half(mb)), __half2float(__ushort_as_half(db)), code);
        uint32_t unit[2], nib[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            unit[e] = (uint32_t)(code[4 * e] | (code[4 * e + 1] << 5) | (code[4 * e + 2] << 10) | ((code[4 * e + 3] >> 4) << 15));
            nib[e] = (uint32_t)code[4 * e + 3] & 15u;
        }
        // nibbles of blocks b and b + 1 share a byte: the even block's lane
        // writes the byte of g = 2c, the odd block's that of g = 2c + 1
        const uint32_t other = __shfl_xor_sync(0xffffffffu, (b & 1) ? nib[0] : nib[1], 4);
        if (on) {
            uint8_t* dm = cell + 864 * NB + (j * NB + b) * 16 + i4 * 2;
            if (c < 2) *reinterpret_cast<unsigned short*>(dm + 8 * c) = c ? mb : db;
            uint8_t* up = cell + 544 * NB + (n >> 2) * 512 + (n & 3) * 4 + s * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<unsigned short*>(up + (4 * (2 * c + e) + j) * 16) = (unsigned short)unit[e];
            const int ne = n & ~1;                 // n is even where b is
            const int g = 2 * c + (b & 1);
            const uint32_t byte = (b & 1) ? (other | (nib[1] << 4)) : (nib[0] | (other << 4));
            cell[800 * NB + (ne >> 2) * 128 + (4 * g + j) * 4 + s * 2 + ((ne & 3) >> 1)] = (uint8_t)byte;
        }
    }
}

// E4M3 rows, many a sequence: pieces of RT rows of one entry that lie at
// RT-aligned positions (RT 8, at head_dim 64 16), so that what a piece holds of V
// in a cell is whole 512-byte stretches.  A CTA takes the pieces whose first row of
// this call is one of its RT rows: at most RT, nearly always one.  A warp's task is
// a piece of one KV head, up to four blocks of K or of V, a lane a block of one
// row; values go through shared memory into 16-byte stores, where append_kernel
// stores them byte by byte.  6 x 1379 rows, 32 query and 8 KV heads of 128: 42 us,
// append_kernel 67 (its q8_0 / q5_1 rows: 48; by pieces they took 56: the exact rounding of
// a whole block a lane is much code).
template <int NB, bool BF16, bool MORE>
__global__ void __launch_bounds__(kCellThreads, BF16 ? 5 : 4) append_cells_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ Freqs fq) {
    constexpr int D = NB * 32, LR = D / 8, BL = NB < 4 ? NB : 4, RT = 32 / BL, W = 2 * RT;
    extern __shared__ float2 s_cs[];                 // [W][rope_dim / 2]
    __shared__ Place s_place[W];
    __shared__ int s_at[MORE ? W : 1][kMaxAxes];     // given positions; -1: the row is skipped
    __shared__ int s_from[W];                        // the piece of a row: index of its first row, -1 none of this CTA's
    __shared__ __align__(16) uint8_t s_stage[kCellWarps][1024];
    constexpr int kSlots = 32;                       // threads that take different pairs
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // every other CTA rotates queries, which HBM bounds, beside those that work codes out
    const bool queries = a.q && (blockIdx.x & 1);
    const int row0 = (a.q ? blockIdx.x >> 1 : blockIdx.x) * RT, half = a.rope_dim / 2;
    wait_for_earlier();
    let_next_start();
    if (warp == 0) {
        const int row = row0 + lane;
        [[maybe_unused]] int at[kMaxAxes] = {};
        if (MORE && a.positions && lane < W && row < a.r.rows) load_positions(a, row, at);
        const int i = entry_of_rows<W>(a.r, row0, lane);
        if (lane < W) {
            Place p{-1, -1, 0, 0, 0};
            if (row < a.r.rows) p = place_in(a.g, a.r, row, i, true);
            const int from = p.pos < 0 ? -1 : queries ? lane : lane - min(p.pos & (RT - 1), p.pos - p.first);
            s_place[lane] = p;
            s_from[lane] = from < RT ? from : -1;    // (below 0: the CTA before has it)
            if (MORE && a.positions && from >= 0 && from < RT) {
                check_positions(a, at);
#pragma unroll
                for (int x = 0; x < kMaxAxes; ++x) s_at[lane][x] = at[x];
            }
        }
    }
    __syncthreads();
    const auto skipped = [&](int i) { return MORE && a.positions && s_at[i][0] < 0; };   // (of rows that are this CTA's)
    // a pair a thread (an indexed read of the frequencies takes a step for each lane), every token
    const int stride_cs = half + 1;                  // rows of the tables start in different banks
    for (int pr = tid % kSlots; pr < half; pr += kSlots) {
        const float2 f = fq.f[pr];
        const int axis = MORE && a.positions ? fq.axis[pr] : 0;
        for (int tt = tid / kSlots; tt < W; tt += kCellThreads / kSlots)
            if (s_from[tt] >= 0) {
                if (MORE && a.positions) put_angle_at(s_cs + tt * stride_cs, f, s_at[tt][axis], pr, half, a.interleaved);
                else put_angle(s_cs + tt * stride_cs, f, s_place[tt].pos, pr, half, a.interleaved);
            }
    }
    const int per = a.g.Hkv * (NB / BL);             // tasks of a piece and kind
    const int li = lane / BL, bl = lane % BL;        // row of the piece, block of the four
    if (queries) {
        __syncthreads();
        for (int i = warp; i < RT; i += kCellWarps)      // a row a warp
            if (s_from[i] >= 0 && !skipped(i)) rotate_queries<LR, BF16>(a, row0 + i, s_cs + i * stride_cs, 0, 1, lane);
        return;
    }
    if (MORE && a.row_scores)
        for (int i = warp; i < W; i += kCellWarps)
            if (s_from[i] >= 0 && s_place[i].cell >= 0 && !skipped(i)) clear_scores(a, s_place[i], lane, 32);
    // values first, for they need no angles
#pragma unroll 1
    for (int kind = 1; kind >= 0; --kind) {
        if (kind == 0) __syncthreads();              // the angles are there
#pragma unroll 1
        for (int s = 0; s < RT; ++s) {
            if (s_from[s] != s) continue;
            // the piece's rows: aligned row li is row s + li - skew of the window
            const Place pf = s_place[s];
            const int skew = pf.pos & (RT - 1), wi = s + li - skew;
            if (pf.cell < 0) continue;
            const bool on = wi >= s && wi < W && s_from[wi] == s && !skipped(wi);
            const bool full = __all_sync(0xffffffffu, on);
            const int t = (pf.pos - skew + li) & 15, j = (t & 7) >> 1, sb = t & 1, hh = t >> 3;
            const long long row = row0 + wi;
            const float2* cs = s_cs + (on ? wi : s) * stride_cs;
            const void* src = kind ? a.v : a.k;
            const long long stride = kind ? a.v_stride : a.k_stride;
#pragma unroll 1
            for (int task = warp; task < per; task += kCellWarps) {
                const int h = task / (NB / BL), b = (task - h * (NB / BL)) * BL + bl, n = hh * NB + b, e0 = 32 * b;
                uint8_t* cell = a.g.pool + pf.cell + (long long)h * a.g.cells_per_page() * a.g.cell_bytes;
                const long long at = row * stride + h * D;
                float x[32];
                {
                    Raw8<BF16> raw[4] = {};
                    if (on)
#pragma unroll
                        for (int k = 0; k < 4; ++k) fetch8(src, at + e0 + 8 * k, raw[k]);
                    Raw8<BF16> other[4] = {};        // what the half-split rotation pairs them with
                    if (on && !kind && !a.interleaved)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int e = e0 + 8 * k;
                            if (e < a.rope_dim) fetch8(src, at + (e < half ? e + half : e - half), other[k]);
                        }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int e = e0 + 8 * k;
                        float v[8], y[8];
                        floats8(raw[k], v);
                        if (!kind && e < a.rope_dim) {
                            floats8(other[k], y);
                            turn8(v, y, e, a.rope_dim, a.interleaved, cs);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[8 * k + i] = v[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = number(x[i]);
                uint32_t w[8];                       // elements 4 g ..
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    w[g] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * g], x[4 * g + 1]), __NV_SATFINITE, __NV_E4M3) |
                           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * g + 2], x[4 * g + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
                if (kind == 0) {
                    // the lanes of blocks b and b + 1 swap halves: 16 bytes hold both blocks' eight of a chunk
                    const bool odd = b & 1;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t g0 = odd ? w[2 * k] : w[4 + 2 * k], g1 = odd ? w[2 * k + 1] : w[5 + 2 * k];
                        const uint32_t m0 = odd ? w[4 + 2 * k] : w[2 * k], m1 = odd ? w[5 + 2 * k] : w[2 * k + 1];
                        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, g0, 1), r1 = __shfl_xor_sync(0xffffffffu, g1, 1);
                        const uint4 v = odd ? make_uint4(r0, r1, m0, m1) : make_uint4(m0, m1, r0, r1);
                        if (on) *reinterpret_cast<uint4*>(cell + (b >> 1) * 1024 + t * 64 + ((odd ? 2 : 0) + k) * 16) = v;
                    }
                    continue;
                }
                if (full) {
                    // rows t and t + 1 alternate byte by byte: their lanes swap halves
                    uint8_t* st = s_stage[warp] + (NB == 2 ? hh : (b >> 1) & 1) * 512 + j * 16 + (n & 1) * 8;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t r = __shfl_xor_sync(0xffffffffu, sb ? w[k] : w[4 + k], BL), m = sb ? w[4 + k] : w[k];
                        const uint32_t even = sb ? r : m, od = sb ? m : r;
                        *reinterpret_cast<uint2*>(st + (k + 4 * sb) * 64) = make_uint2(__byte_perm(even, od, 0x5140), __byte_perm(even, od, 0x7362));
                    }
                    __syncwarp();
                    // regions n >> 1: of NB 2 the cell's two, else this half's pair of pairs
                    uint8_t* dst = cell + 512 * NB + (NB == 2 ? 0 : (hh * NB + b - bl) / 2 * 512);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(dst + 512 * k + lane * 16) = *reinterpret_cast<const uint4*>(s_stage[warp] + 512 * k + lane * 16);
                    __syncwarp();
                } else if (on) {
                    uint8_t* p = cell + 512 * NB + (n >> 1) * 512 + (n & 1) * 8 + sb;
#pragma unroll
                    for (int i = 0; i < 32; ++i) p[(4 * (i >> 2) + j) * 16 + (i & 3) * 2] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
                }
            }
        }
    }
}

// The 8 elements of lane li's K (or V) of row t of a cell, as f32
template <int NB>
__device__ __forceinline__ void read_k8(const uint8_t* cell, int fp8, int t, int b, int c, float (&x)[8]) {
    const uint2 w = *reinterpret_cast<const uint2*>(cell + (b >> 1) * 1024 + t * 64 + c * 16 + (b & 1) * 8);
    const uint32_t w2[2] = {w.x, w.y};
    if (fp8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((w2[i >> 2] >> (8 * (i & 3))) & 255u, __NV_E4M3)));
        return;
    }
    const int j = (t & 7) >> 1, i4 = 2 * (t >> 3) + (t & 1);
    const float d = __half2float(*reinterpret_cast<const __half*>(cell + 512 * NB + (j * NB + b) * 8 + i4 * 2));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((int)((w2[i >> 2] >> (8 * (i & 3))) & 255u) - 128) * d;
}

template <int NB>
__device__ __forceinline__ void read_v8(const uint8_t* cell, int fp8, int t, int b, int c, float (&x)[8]) {
    const int j = (t & 7) >> 1, s = t & 1, hh = t >> 3, n = hh * NB + b, i4 = 2 * hh + s;
    if (fp8) {
        const uint8_t* p = cell + 512 * NB + (n >> 1) * 512 + (n & 1) * 8 + s;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(p[(4 * (2 * c + (i >> 2)) + j) * 16 + (i & 3) * 2], __NV_E4M3)));
        return;
    }
    const uint8_t* dm = cell + 864 * NB + (j * NB + b) * 16 + i4 * 2;
    const float d = __half2float(*reinterpret_cast<const __half*>(dm)), m = __half2float(*reinterpret_cast<const __half*>(dm + 8));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int ln = 4 * (2 * c + e) + j;
        const uint32_t unit = *reinterpret_cast<const unsigned short*>(cell + 544 * NB + (n >> 2) * 512 + ln * 16 + (n & 3) * 4 + s * 2);
        const uint32_t nb = (cell[800 * NB + (n >> 2) * 128 + ln * 4 + s * 2 + ((n & 3) >> 1)] >> (4 * (n & 1))) & 15u;
        const uint32_t u[4] = {unit & 31u, (unit >> 5) & 31u, (unit >> 10) & 31u, ((unit >> 15) << 4) | nb};
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * e + r] = fmaf((float)u[r], d, m);
    }
}

// Rows back as values: LR lanes a (row, KV head), K and V both.  8k rows of 8 KV heads
// of 128 to bf16: 17 us (10 of bytes).
template <int LR>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a) {
    constexpr int D = LR * 8, NB = D / 32;
    wait_for_earlier();
    let_next_start();
    const long long w = (long long)blockIdx.x * (kThreads / LR) + threadIdx.x / LR;
    const int row = (int)(w / a.g.Hkv), h = (int)(w - (long long)row * a.g.Hkv);
    if (row >= a.r.rows) return;
    const Place p = place_row(a.g, a.r, row, false);
    if (a.r.starts && (row < a.r.starts[0] || row >= a.r.starts[a.r.n_seq])) return;
    const int li = threadIdx.x % LR, b = li >> 2, c = li & 3;
    float k[8] = {}, v[8] = {};
    if (p.cell >= 0) {
        const uint8_t* cell = a.g.pool + p.cell + (long long)h * a.g.cells_per_page() * a.g.cell_bytes;
        read_k8<NB>(cell, a.g.fp8, p.t, b, c, k);
        read_v8<NB>(cell, a.g.fp8, p.t, b, c, v);
    }
    const long long at = ((long long)row * a.g.Hkv + h) * D + 8 * li;
    store8(a.k_out, at, a.bf16, k);
    store8(a.v_out, at, a.bf16, v);
}

// Key bounds: one warp per (row, KV head, pair of blocks) whose row is the
// first of this call in its page; it goes over the page's rows below the length
// 8 at a time (lane = row in the eight, 16 elements).  A warp of another row has nothing to do.
template <int NB>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const BoundsArgs a) {
    wait_for_earlier();
    let_next_start();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = a.g.Hkv * (NB / 2);
    const int row = (int)(w / per), rest = (int)(w - (long long)row * per);
    const int h = rest / (NB / 2), bp = rest - h * (NB / 2);
    if (row >= a.r.rows) return;
    const Place p = place_row(a.g, a.r, row, false);
    if (p.cell < 0) return;
    const int in = p.pos & (a.g.page_rows - 1);
    if (in != 0 && p.pos != p.first) return;
    const int valid = min(a.g.page_rows, p.len - (p.pos - in));
    const long long page = (p.cell - (long long)(in >> 4) * a.g.cell_bytes) / a.g.page_bytes;
    const uint8_t* cell0 = a.g.pool + page * a.g.page_bytes + (long long)h * a.g.cells_per_page() * a.g.cell_bytes;
    const int g8 = lane >> 2, c = lane & 3;
    float mn[16], mx[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        mn[i] = __builtin_huge_valf();
        mx[i] = -__builtin_huge_valf();
    }
    for (int r = g8; r < valid; r += 8) {
        const uint8_t* cell = cell0 + (long long)(r >> 4) * a.g.cell_bytes;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x[8];
            read_k8<NB>(cell, a.g.fp8, r & 15, 2 * bp + e, c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mn[8 * e + i] = fminf(mn[8 * e + i], x[i]);
                mx[8 * e + i] = fmaxf(mx[8 * e + i], x[i]);
            }
        }
    }
    float am[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            mn[i] = fminf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], o));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
        }
        am[i >> 3] = fmaxf(am[i >> 3], fmaxf(fabsf(mn[i]), fabsf(mx[i])));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        am[e] = fmaxf(am[e], __shfl_xor_sync(0xffffffffu, am[e], 1));
        am[e] = fmaxf(am[e], __shfl_xor_sync(0xffffffffu, am[e], 2));
        const int b = 2 * bp + e;
        const float ds = __fmul_rn(am[e], 1.0f / 127.0f);
        const long long at = (page * a.g.Hkv + h) * NB + b;
        if (g8 == 0) store_bounds(a.codes, a.scales, at, c, ds, &mn[8 * e], &mx[8 * e]);
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, const Freqs& f, int num_sms, cudaStream_t s) {
    const std::true_type yes;
    const std::false_type no;
    const bool more = a.positions || a.row_scores;
    // pieces of cells where a sequence brings 8 rows or more on average
    if (a.g.fp8 && a.r.rows / 8 >= a.r.n_seq) {
        const int rt = a.g.D == 64 ? 16 : 8;
        const dim3 grid((unsigned)((a.r.rows + rt - 1) / rt * (a.q ? 2 : 1)));
        const size_t smem = (size_t)2 * rt * (a.rope_dim / 2 + 1) * sizeof(float2);
        auto run = [&](auto b, auto with_more) {
            constexpr bool B = decltype(b)::value, M = decltype(with_more)::value;
            if (a.g.D == 64) return launch_dependent(append_cells_kernel<2, B, M>, grid, kCellThreads, smem, s, a, f);
            if (a.g.D == 128) return launch_dependent(append_cells_kernel<4, B, M>, grid, kCellThreads, smem, s, a, f);
            return launch_dependent(append_cells_kernel<8, B, M>, grid, kCellThreads, smem, s, a, f);
        };
        if (more) return a.bf16 ? run(yes, yes) : run(no, yes);
        return a.bf16 ? run(yes, no) : run(no, no);
    }
    const int jpw = 256 / a.g.D, qpw = 2 * jpw;
    const int units = (a.q ? (a.Hq + qpw - 1) / qpw : 0) + 2 * ((a.g.Hkv + jpw - 1) / jpw);
    // tokens per CTA: the angles are shared by its heads; few rows spread over
    // the SMs by heads instead
    const int TT = a.r.rows >= 16 * num_sms ? kTT : a.r.rows >= 4 * num_sms ? 2 : 1;
    const int gx = (a.r.rows + TT - 1) / TT;
    const int most = (units * TT + kWarps - 1) / kWarps;
    const int gy = std::max(1, std::min(most, (2 * num_sms + gx - 1) / gx));
    const size_t smem = (size_t)TT * (a.rope_dim / 2) * sizeof(float2);
    const dim3 grid((unsigned)gx, (unsigned)gy);
    auto run = [&](auto b, auto with_bounds, auto with_more) {
        constexpr bool B = decltype(b)::value, W = decltype(with_bounds)::value, M = decltype(with_more)::value;
        if (a.g.D == 64) return launch_dependent(append_kernel<8, B, W, M>, grid, kThreads, smem, s, a, f, TT);
        if (a.g.D == 128) return launch_dependent(append_kernel<16, B, W, M>, grid, kThreads, smem, s, a, f, TT);
        return launch_dependent(append_kernel<32, B, W, M>, grid, kThreads, smem, s, a, f, TT);
    };
    if (more) {
        if (a.codes) return a.bf16 ? run(yes, yes, yes) : run(no, yes, yes);
        return a.bf16 ? run(yes, no, yes) : run(no, no, yes);
    }
    if (a.codes) return a.bf16 ? run(yes, yes, no) : run(no, yes, no);
    return a.bf16 ? run(yes, no, no) : run(no, no, no);
}

cudaError_t launch_read(const ReadArgs& a, cudaStream_t s) {
    const int lr = a.g.D / 8;
    const long long groups = (long long)a.r.rows * a.g.Hkv;
    const unsigned grid = (unsigned)((groups + kThreads / lr - 1) / (kThreads / lr));
    if (lr == 8) return launch_dependent(read_kernel<8>, dim3(grid), kThreads, 0, s, a);
    if (lr == 16) return launch_dependent(read_kernel<16>, dim3(grid), kThreads, 0, s, a);
    return launch_dependent(read_kernel<32>, dim3(grid), kThreads, 0, s, a);
}

cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t s) {
    const int nb = a.g.NB();
    const long long warps = (long long)a.r.rows * a.g.Hkv * (nb / 2);
    const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
    if (nb == 2) return launch_dependent(bounds_kernel<2>, dim3(grid), kThreads, 0, s, a);
    if (nb == 4) return launch_dependent(bounds_kernel<4>, dim3(grid), kThreads, 0, s, a);
    return launch_dependent(bounds_kernel<8>, dim3(grid), kThreads, 0, s, a);
}

}  // namespace paged
}  // namespace kvq
