// The shared part of kvq_paged_decode_shared for groups with more queries than
// one 16-row tile: tcgen05 matrix products over 128-row tiles of the prefix.
//
// Mathematics: as the split kernel's (one pass over the rows, a reference that
// moves when a score passes it by 8), for up to 256 queries at once (two tiles
// of 128; one at head_dim 256, whose output takes the tensor memory of two):
//   S = Q K^T   (M 128 queries, N 128 rows, K head_dim), f32 in tensor memory;
//   P = 2^(s - m), fp16, written over S;
//   O += P V    (A operand P from tensor memory), f32 in tensor memory.
// K and V are turned from codes into fp16 tiles in shared memory once for all
// queries: K as (d 2^s) (c 2^-8), both factors exact and one rounding, with s of
// each 32 rows such that their largest d 2^s lies in [2^15, 2^16): no key overflows,
// and one of 2^-28 of the largest still has its 11 bits (a fixed power would leave
// keys around 1e-4 four of them); 2^(8 - s) joins the score's factor.  V as u d + m
// (one rounding).
// Both tiles are K-major in the 128-byte swizzle; the rows of a tile are taken in
// the order in which a lane of the unpacking warps holds them (of 32 rows, place
// p is row 16 (p/4 % 2) + 8 (p/2 % 2) + 2 (p/8) + p % 2), which makes each lane's
// pieces whole 16-byte chunks in different banks; sums do not depend on it.
//
// Roles in a CTA (one an SM): 4 or 8 softmax warps (a query row a thread), 8
// unpacking warps (four pairs of cells, K or V of one each), one warp that issues
// the products.  With two query tiles the products of one run while the
// exponentials of the other are worked out.
//
// Bound: a row of head_dim 128 costs 232 bytes of HBM a KV head and 512 flops a
// query, so at the measured rates (6.8 TB/s, 1.9 PFLOP/s) the products cost what the
// bytes cost from about 130 queries a KV head on.  Measured: 8192 rows for 64
// sequences of 4 queries a KV head, 8 KV heads of 128: 27 us for 3.4 tiles an SM
// (the products 4.4 us at cuBLAS's rate), tensor cores 13 % busy: half is before the
// first products and after the last, and a tile's products wait for its softmax.
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

constexpr int kTileRows = 128;
constexpr int kUnpackWarps = 8;

template <int NB>
struct Shape {
    static constexpr int D = NB * 32;
    static constexpr int QT = NB == 8 ? 1 : 2;                 // query tiles of 128
    static constexpr int ST = NB == 8 ? 1 : 2;                 // K/V stages
    static constexpr int kSoftWarps = 4 * QT;
    static constexpr int kWarps = kSoftWarps + kUnpackWarps + 1;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int tile = kTileRows * D * 2;             // bytes of a K, V or Q tile
    static constexpr size_t smem = (size_t)QT * tile + (size_t)ST * 2 * tile + 1024;
};

struct Barriers {
    uint64_t q_ready, s_full[2], p_ready[2], o_done[2], kv_full[2], kv_free[2];
};

// ------------------------------------------------------------ tcgen05

// K-major operand tile in the 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// f16 x f16 -> f32, both K-major
__host__ __device__ constexpr uint32_t instr_desc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N / 8) << 17) | ((uint32_t)(M / 16) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
        "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------ unpacking

// One warp's raw bytes of a pair of cells, K or V, of up to four blocks, in the
// order in which they are used: the unpacking is a rolled loop that takes the
// front words and shifts the rest down.  (Unrolled, the code of a tile is some
// 20 KB, and fetching that for the first tile took 5 us.)
//   K: for each block pair and cell, 8 words of codes (rows g, g + 8 of the cell)
//      and 4 of scales;  V: for each block, 4 words of units (cell, half) and 8 of
//      d, m, then 4 words of nibbles;  E4M3: 8 words of bytes each.
template <int NBT, bool F8>
struct Raw {
    uint32_t w[F8 ? 8 * NBT : 12 * NBT], nib[4];
    template <int N>
    __device__ __forceinline__ void shift() {
#pragma unroll
        for (int i = 0; i + N < (F8 ? 8 * NBT : 12 * NBT); ++i) w[i] = w[i + N];
    }
};

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// b0: first block of the task
template <int NB, int NBT, bool F8>
__device__ __forceinline__ void load_k(const uint8_t* c0, const uint8_t* c1, int b0, int lane, Raw<NBT, F8>& r) {
    constexpr int N = F8 ? 8 : 12;
    const int g = lane >> 2;
#pragma unroll
    for (int bp = 0; bp < NBT / 2; ++bp)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint8_t* cell = c ? c1 : c0;
            uint32_t* w = r.w + (2 * bp + c) * N;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (cell) x = ldg16(cell + (b0 / 2 + bp) * 1024 + t * 512 + lane * 16);
                w[4 * t] = x.x; w[4 * t + 1] = x.y; w[4 * t + 2] = x.z; w[4 * t + 3] = x.w;
            }
            if constexpr (!F8) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (cell) x = ldg16(cell + 512 * NB + ((g >> 1) * NB + b0 + 2 * bp) * 8);
                w[8] = x.x; w[9] = x.y; w[10] = x.z; w[11] = x.w;   // d of rows (g & ~1, + 1), then + 8; two blocks
            }
        }
}
template <int NB, int NBT, bool F8>
__device__ __forceinline__ void load_v(const uint8_t* c0, const uint8_t* c1, int b0, int lane, Raw<NBT, F8>& r) {
    const int j = lane & 3;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint8_t* cell = c ? c1 : c0;
        if constexpr (F8) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NBT / 2; ++i) {           // blocks 2i, 2i + 1 of half h
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (cell) x = ldg16(cell + 512 * NB + ((h * NB + b0) / 2 + i) * 512 + lane * 16);
                    uint32_t* w = r.w + 16 * i + 4 * c + 2 * h;
                    w[0] = x.x; w[1] = x.y; w[8] = x.z; w[9] = x.w;
                }
        } else {
            // units (h NB + b), 4 a chunk: with two blocks one chunk holds both
            // halves, else each half has its own
#pragma unroll
            for (int h = 0; h < (NB == 2 ? 1 : 2); ++h) {
                const int n = NB == 2 ? 0 : h * NB + b0;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                uint32_t e = 0u;
                if (cell) {
                    x = ldg16(cell + 544 * NB + (n / 4) * 512 + lane * 16);
                    e = *reinterpret_cast<const uint32_t*>(cell + 800 * NB + (n / 4) * 128 + lane * 4);
                }
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int b = NB == 2 ? (i & 1) : i, hh = NB == 2 ? (i >> 1) : h;
                    r.w[12 * b + 2 * c + hh] = u[i];
                }
                r.nib[2 * c + h] = e;
                if (NB == 2) r.nib[2 * c + 1] = e >> 8;
            }
#pragma unroll
            for (int b = 0; b < NBT; ++b) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (cell) x = ldg16(cell + 864 * NB + (j * NB + b0 + b) * 16);
                uint32_t* w = r.w + 12 * b + 4 + 4 * c;
                w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            }
        }
    }
}

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The scales d of a pair of cells, words of two rows: index w of a cell's 8 NB words
// is rows 8 (w % 2) + 2 (w / (2 NB)) and + 1 of block w / 2 % NB.
template <int NB>
struct Scales {
    static constexpr int N = NB == 8 ? 2 : 1;                 // words of a lane (NB 2: half of the lanes)
    uint32_t w[2][N];
    __device__ __forceinline__ void load(const uint8_t* c0, const uint8_t* c1, int lane) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint8_t* cell = c ? c1 : c0;
                const int at = lane + 32 * i;
                w[c][i] = 0u;
                if (cell && at < 8 * NB) w[c][i] = *reinterpret_cast<const uint32_t*>(cell + 512 * NB + 4 * at);
            }
    }
    // s by the largest finite d of the pair's first `rows` rows (those behind may be any bytes)
    __device__ __forceinline__ int shift(int rows, int lane) const {
        uint32_t top = 0u;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = lane + 32 * i, r = 16 * c + 8 * (at & 1) + 2 * (at / (2 * NB));
                const uint32_t a = w[c][i] & 0x7fffu, b = (w[c][i] >> 16) & 0x7fffu;
                if (r < rows && a < 0x7c00u) top = max(top, a);
                if (r + 1 < rows && b < 0x7c00u) top = max(top, b);
            }
        return 30 - (int)(__reduce_max_sync(0xffffffffu, top) >> 10);
    }
};
// 2^e as a half pair, 0 <= e <= 15
__device__ __forceinline__ __half2 pow2_pair(int e) { return as_h2((uint32_t)(15 + e) * 0x04000400u); }

// K tile: rows of head_dim / 64 column blocks of 128 bytes; pr: the pair of cells,
// shift: their s, 0 .. 30
template <int NB, int NBT, bool F8>
__device__ __forceinline__ void store_k(uint32_t tile, int pr, int b0, int lane, int shift, Raw<NBT, F8>& r) {
    const int g = lane >> 2, j = lane & 3;
    const uint32_t dsel = (g & 1) ? 0x3232u : 0x1010u, exps = held(0x44444444u);
    const __half2 up0 = pow2_pair(min(shift, 15)), up1 = pow2_pair(max(shift - 15, 0));
#pragma unroll 1
    for (int it = 0; it < NBT; ++it) {                        // block pair it / 2, cell it % 2
        const int row0 = 32 * pr + 8 * (g >> 1) + 4 * (it & 1) + (g & 1);
        const uint32_t base = tile + (b0 / 2 + (it >> 1)) * (kTileRows * 128);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = row0 + 2 * t;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t x = r.w[4 * t + 2 * e], y = r.w[4 * t + 2 * e + 1];
                uint32_t o[4];
                if constexpr (F8) {
                    o[0] = f8_pair(x);
                    o[1] = f8_pair(x >> 16);
                    o[2] = f8_pair(y);
                    o[3] = f8_pair(y >> 16);
                } else {
                    const __half2 dd = __hmul2(__hmul2(as_h2(__byte_perm(r.w[8 + 2 * e + t], 0, dsel)), up0), up1);
                    auto two = [&](uint32_t v, uint32_t sel) {
                        return as_u32(__hmul2(__hsub2(as_h2(__byte_perm(v, exps, sel)), as_h2(0x44804480u)), dd));
                    };
                    o[0] = two(x, 0x4140u);
                    o[1] = two(x, 0x4342u);
                    o[2] = two(y, 0x4140u);
                    o[3] = two(y, 0x4342u);
                }
                sts16(base + row * 128 + (((4 * e + j) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
            }
        }
        r.template shift<F8 ? 8 : 12>();
    }
}
// V tile: rows are elements, columns the tile's rows, 64 a block of 128 bytes.
// keep: half-word masks of the lane's rows (2j, 2j+1 | 2j+8, 2j+9) of both cells
template <int NB, int NBT, bool F8>
__device__ __forceinline__ void store_v(uint32_t tile, int pr, int b0, int lane, const uint32_t (&keep)[4], Raw<NBT, F8>& r) {
    constexpr int D = NB * 32;
    const int g = lane >> 2, j = lane & 3;
    const uint32_t block = tile + (pr >> 1) * (D * 128);
    const int chunk = 4 * (pr & 1) + j;
    const uint32_t magic = held(0x64006400u);
#pragma unroll 1
    for (int b = 0; b < NBT; ++b) {
        uint32_t o[4][4];                                     // element r, (cell, half)
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
            const uint32_t k = keep[ch];
            if constexpr (F8) {
                const uint32_t kb = __byte_perm(k, 0, 0x2020);
                const uint32_t x = r.w[2 * ch] & kb, y = r.w[2 * ch + 1] & kb;
                o[0][ch] = f8_pair(x);
                o[1][ch] = f8_pair(x >> 16);
                o[2][ch] = f8_pair(y);
                o[3][ch] = f8_pair(y >> 16);
            } else {
                const uint32_t unit = r.w[ch], nib = r.nib[ch];
                const uint32_t* dm = r.w + 4 + 4 * (ch >> 1);
                const __half2 d = as_h2(dm[ch & 1] & k), m = as_h2(dm[2 + (ch & 1)] & k);
                auto val = [&](auto R) {
                    const __half2 u = __hsub2(as_h2(v_codes<decltype(R)::value>(unit, nib, 0, magic)), as_h2(magic));
                    return as_u32(__hfma2(u, d, m));
                };
                o[0][ch] = val(std::integral_constant<int, 0>{});
                o[1][ch] = val(std::integral_constant<int, 1>{});
                o[2][ch] = val(std::integral_constant<int, 2>{});
                o[3][ch] = val(std::integral_constant<int, 3>{});
                r.nib[ch] = nib >> 4;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 32 * (b0 + b) + 4 * g + i;
            sts16(block + row * 128 + ((chunk ^ (row & 7)) << 4), o[i][0], o[i][1], o[i][2], o[i][3]);
        }
        r.template shift<F8 ? 8 : 12>();
    }
}

// Places of a 32-row group whose rows lie in [lo, hi) and whose cells (bits of
// there) are present: the row mask with index bits 4 and 2, 3 and 1 exchanged
__device__ __forceinline__ uint32_t seen_places(int lo, int hi, int there) {
    lo = min(max(lo, 0), 32);
    hi = min(max(hi, 0), 32);
    uint32_t m = (hi >= 32 ? 0xffffffffu : (1u << hi) - 1u) & ~(lo >= 32 ? 0xffffffffu : (1u << lo) - 1u);
    m &= ((there & 1) ? 0x0000ffffu : 0u) | ((there & 2) ? 0xffff0000u : 0u);
    uint32_t t = ((m >> 12) ^ m) & 0x0000f0f0u;              // index bits 4 and 2
    m ^= t ^ (t << 12);
    t = ((m >> 6) ^ m) & 0x00cc00ccu;                        // index bits 3 and 1
    return m ^ t ^ (t << 6);
}

// ------------------------------------------------------------ the kernel

// A CTA's part of a key: group, KV head, query block qb, tiles [ta, tb)
struct Part {
    int kh, qb, nqb, nq, gs, t0, ta, tb, kk, keys, hi;     // gs: first member; hi: rows of the prefix that are seen
};

template <int NB, bool F8>
__global__ void __launch_bounds__(Shape<NB>::kThreads, 1) prefix_kernel(const __grid_constant__ SplitArgs a) {
    using S = Shape<NB>;
    constexpr int D = S::D, QT = S::QT, ST = S::ST, QB = 128 * QT;
    constexpr int NBT = NB == 2 ? 2 : 4, NQ4 = NB / NBT;       // blocks of an unpacking task, tasks a pair of cells
    constexpr uint32_t kSCols = 128, kOCol = QT * kSCols;      // S / P of tile q at column 128 q, O at kOCol + D q
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Barriers bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_ok[2][4];                                 // of each pair of a stage: cells that were there (two bits), s << 2
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (dev::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_tile = base, kv_tile = base + QT * S::tile;

    if (tid == 0) {
        s_abort = 0;
        dev::mbar_init(dev::smem_u32(&bars.q_ready), S::kSoftWarps);
        for (int q = 0; q < 2; ++q) {
            dev::mbar_init(dev::smem_u32(&bars.s_full[q]), 1);
            dev::mbar_init(dev::smem_u32(&bars.p_ready[q]), 4);
            dev::mbar_init(dev::smem_u32(&bars.o_done[q]), 1);
            dev::mbar_init(dev::smem_u32(&bars.kv_full[q]), kUnpackWarps);
            dev::mbar_init(dev::smem_u32(&bars.kv_free[q]), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_earlier();
    // ---- the plan: a warp a group (the rows its members see of the prefix), then
    // a scan by one warp; CTA 0 keeps it for the merge
    PlanEntry* plan = reinterpret_cast<PlanEntry*>(smem_raw + (base - dev::smem_u32(smem_raw)) + (QT + 2 * ST) * S::tile);
    for (int grp = warp; grp < a.n_groups; grp += S::kWarps) {
        int gs, ge;
        members(a, grp, gs, ge);
        const int nq = (ge - gs) * a.hpk * a.T, pre = prefix_rows(a, grp);
        int lo = a.window > 0 ? pre : 0, hi = 0;
        for (int s = gs + lane; s < ge; s += 32) {
            const int len = a.lens[s];
            if (!len_ok(a, len)) continue;
            hi = max(hi, len);
            if (a.window > 0) lo = min(lo, max(0, len - a.T + 1 - a.window));
        }
        hi = min(pre, __reduce_max_sync(0xffffffffu, hi));
        lo = __reduce_min_sync(0xffffffffu, lo);
        if (lane == 0) {
            PlanEntry pe{};
            if (tile_group(a, nq) && hi > lo) {
                pe.c0 = lo / kTileRows;
                pe.nc = (hi + kTileRows - 1) / kTileRows - pe.c0;
                pe.nq = nq;
                pe.rows = hi;
                pe.lo = gs;
            }
            plan[grp] = pe;
        }
    }
    __syncthreads();
    if (warp == 0) {
        long long w = 0;
        int k = 0;
        for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
            const int grp = g0 + lane;
            const int nqb = grp < a.n_groups ? (plan[grp].nq + QB - 1) / QB : 0;
            const long long own = grp < a.n_groups ? (long long)plan[grp].nc * nqb : 0;
            long long wi = own;
            int ki = nqb;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, wi, o);
                const int z = __shfl_up_sync(0xffffffffu, ki, o);
                if (lane >= o) {
                    wi += y;
                    ki += z;
                }
            }
            if (grp < a.n_groups) {
                plan[grp].work = w + wi - own;
                plan[grp].keys = k + ki - nqb;
            }
            w += __shfl_sync(0xffffffffu, wi, 31);
            k += __shfl_sync(0xffffffffu, ki, 31);
        }
        if (lane == 0) {
            const bool fits = (long long)k * a.g.Hkv <= a.max_keys2;
            if (!fits) atomicExch(a.g.err, kErrCounter);
            PlanEntry pe{};
            pe.work = fits ? w : 0;
            pe.keys = k;
            plan[a.n_groups] = pe;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.n_groups; e += S::kThreads) a.plan2[e] = plan[e];
    let_next_start();
    const long long W = plan[a.n_groups].work * a.g.Hkv;
    const int G = (int)min((long long)a.G, W);
    if ((int)blockIdx.x >= G) return;
    if (warp == S::kWarps - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_u32(&s_tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    const long long x1 = W * (blockIdx.x + 1) / G;
    volatile int* abort_flag = &s_abort;
    auto wait = [&](uint64_t& bar, uint32_t parity) { return wait_bounded(dev::smem_u32(&bar), parity, abort_flag, a.g.err); };
    auto part_at = [&](long long x) {
        Part p;
        const PlanEntry pe = plan[find_entry(plan, a.n_groups, x / a.g.Hkv)];
        const long long rel = x - pe.work * a.g.Hkv;
        p.kk = (int)(rel / pe.nc);
        p.ta = (int)(rel - (long long)p.kk * pe.nc);
        p.tb = (int)min((long long)pe.nc, p.ta + (x1 - x));
        p.nq = pe.nq;
        p.nqb = (p.nq + QB - 1) / QB;
        p.kh = p.kk / p.nqb;
        p.qb = p.kk - p.kh * p.nqb;
        p.t0 = pe.c0;
        p.keys = pe.keys;
        p.gs = pe.lo;
        p.hi = pe.rows;
        return p;
    };
    const long long xs = W * blockIdx.x / G;

    if (warp < S::kSoftWarps) {
        // ================= softmax: thread = query row of tile qt
        const int qt = warp >> 2, wr = warp & 3, row = wr * 32 + lane;
        const uint32_t lanes = (uint32_t)(wr * 32) << 16;
        const uint32_t s_addr = tmem + lanes + qt * kSCols, o_addr = tmem + lanes + kOCol + qt * D;
        uint32_t n_tile = 0, n_part = 0;
        int tile_no = 0;                                       // tiles since the start, for the stages
        bool ok = true;
        for (long long x = xs; x < x1 && ok; ++n_part) {
            const Part p = part_at(x);
            x += p.tb - p.ta;
            const int qi = p.qb * QB + qt * 128 + row;
            const bool valid = qi < p.nq, tile_on = p.qb * QB + qt * 128 < p.nq;
            int ex = 0;                                        // the query times 2^-ex is in the tile
            bool bad = false;
            int lo = 0, hi = 0x7fffffff;
            {
                // the query, scaled by a power of two to a largest element in [512, 1024), as fp16
                const int Qh = a.hpk * a.T, seq = p.gs + (valid ? qi / Qh : 0), in = valid ? qi % Qh : 0, tq = in / a.hpk;
                const uint4* src = reinterpret_cast<const uint4*>(
                    reinterpret_cast<const uint16_t*>(a.q) + (((long long)seq * a.T + tq) * a.Hq + p.kh * a.hpk + in - tq * a.hpk) * D);
                const int len = a.lens[seq];
                constexpr int PER = 8;                         // 16-byte pieces in registers at once
                uint4 v[PER];
                auto load = [&](int i0) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) v[i] = valid ? src[i0 + i] : make_uint4(0u, 0u, 0u, 0u);
                };
                uint32_t am = 0u;                              // bits of the largest |element|: NaN above infinity
#pragma unroll 1
                for (int i0 = D / 8 - PER; i0 >= 0; i0 -= PER) {
                    load(i0);
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            am = max(am, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
                    }
                }
                if (valid) {
                    const int end = (len_ok(a, len) ? len : 0) - a.T + tq + 1;
                    hi = min(end, p.hi);
                    lo = a.window > 0 ? max(0, end - a.window) : 0;
                }
                bad = am >= kInfBits;
                ex = am > 0u && !bad ? min(max((int)(am >> 23) - 127 - 9, -117), 118) : 0;
                const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
                const uint32_t dst = q_tile + qt * S::tile + row * 128;
#pragma unroll 1
                for (int i0 = 0; i0 < D / 8; i0 += PER) {
                    if (i0 > 0) load(i0);
#pragma unroll
                    for (int k = 0; k < PER; ++k) {
                        const int i = i0 + k;
                        const uint32_t keep = bad ? 0u : 0xffffffffu;
                        const uint32_t w[4] = {v[k].x & keep, v[k].y & keep, v[k].z & keep, v[k].w & keep};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = as_u32(__floats2half2_rn(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up));
                        sts16(dst + (i >> 3) * (kTileRows * 128) + (((i & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(dev::smem_u32(&bars.q_ready));
                if (!tile_on) {                                // nothing else keeps this warp from arriving twice
                    ok = wait(bars.q_ready, n_part & 1u);
                    if (!ok) break;
                }
            }
            float m = kNone, l = 0.f;
            for (int t = p.ta; t < p.tb && ok; ++t, ++tile_no) {
                if (!tile_on) continue;
                ok = wait(bars.s_full[qt], n_tile & 1u);
                if (!ok) break;
                fence_after();
                const int row0 = (p.t0 + t) * kTileRows;
                const int* okc = s_ok[tile_no % ST];
                const int all = okc[0] & okc[1] & okc[2] & okc[3] & 3;
                const bool masked = __any_sync(0xffffffffu, row0 < lo || row0 + kTileRows > hi || all != 3);
                const bool capped = a.softcap_b > 0.f;
                // Two passes over the scores in 32-column pieces: the largest, then
                // the probabilities.  Capped or masked scores are worked out in
                // both, in log2 units; plain ones enter as they are (the factor is
                // positive) and meet it in the exponent's fma.  A piece is a pair of
                // cells, with its own power of two in the factor.  Where the reference
                // is so large that its last bits show in the fma's exact product (2^-24
                // of it; from 2^27 on p would overflow), plain scores are rounded first.
                float top = dev::kNegInf, add = 0.f, l0 = 0.f, l1 = 0.f;
                bool large = false;
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_ld32(s_addr + 32 * c, r);
                        tmem_wait_ld();
                        const int e2 = max(F8 ? ex : ex + 8 - (okc[c] >> 2), -126);
                        const float fc = factor(a.qscale * __uint_as_float((uint32_t)(127 + e2) << 23));
                        const float f0 = capped || large ? 1.f : fc;
                        if (capped) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[i] = __float_as_uint(a.softcap_b * tanhf(a.softcap_a * (__uint_as_float(r[i]) * fc)));
                        } else if (large) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * fc);
                        }
                        if (masked) {
                            const uint32_t see = seen_places(lo - row0 - 32 * c, hi - row0 - 32 * c, okc[c]);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((see >> i) & 1u)) r[i] = 0xff800000u;
                        }
                        if (pass == 0) {
                            float most = dev::kNegInf;
#pragma unroll
                            for (int i = 0; i < 32; ++i) most = fmaxf(most, __uint_as_float(r[i]));
                            top = fmaxf(top, most * f0);
                        } else {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float p0 = ex2(fmaf(__uint_as_float(r[2 * i]), f0, add));
                                const float p1 = ex2(fmaf(__uint_as_float(r[2 * i + 1]), f0, add));
                                l0 += p0;
                                l1 += p1;
                                pk[i] = as_u32(__floats2half2_rn(p0, p1));
                            }
                            tmem_st16(s_addr + 16 * c, pk);    // over columns that have been read
                        }
                    }
                    if (pass == 1) break;
                    const bool move = top > m + dev::kLazy;
                    if (__any_sync(0xffffffffu, move)) {
                        const float al = move ? ex2(m - top) : 1.f;
                        if (move) m = top;
                        l *= al;
                        if (t > p.ta) {                        // O holds the tiles before: scale it between its products
                            ok = wait(bars.o_done[qt], (n_tile - 1) & 1u);
                            if (!ok) break;
                            fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t r[32];
                                tmem_ld32(o_addr + 32 * c, r);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * al);
                                tmem_st32(o_addr + 32 * c, r);
                                tmem_wait_st();
                            }
                        }
                    }
                    add = kShift - m;
                    large = __any_sync(0xffffffffu, fabsf(m) > 1048576.f && m != kNone);
                }
                if (!ok) break;
                l += l0 + l1;
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(dev::smem_u32(&bars.p_ready[qt]));
                ++n_tile;
            }
            if (!ok) break;
            if (tile_on) {
                // ---- the record: O, reference and sum of this query
                ok = wait(bars.o_done[qt], (n_tile - 1) & 1u);
                if (!ok) break;
                fence_after();
                const long long slot = blockIdx.x + (long long)p.keys * a.g.Hkv + p.kk;
                const long long at = slot * QB + qt * 128 + row;
                // fp16 records hold O times the power of two that brings its largest
                // element into [2^14, 2^15): eleven bits for each that is not below 2^-28
                // of it, where O / l would leave values around 1e-5 few
                float most = 0.f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld32(o_addr + 32 * c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) most = fmaxf(most, fabsf(__uint_as_float(r[i])));
                }
                const uint32_t ue = min(268u - (__float_as_uint(most) >> 23), 253u);
                const float inv = __uint_as_float(ue << 23), back = __uint_as_float((254u - ue) << 23);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld32(o_addr + 32 * c, r);
                    tmem_wait_ld();
                    if (valid) {
                        uint4* dst = reinterpret_cast<uint4*>(a.part2_o + at * D + 32 * c);
                        auto two = [&](int i) { return as_u32(__floats2half2_rn(__uint_as_float(r[i]) * inv, __uint_as_float(r[i + 1]) * inv)); };
#pragma unroll
                        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(two(8 * i), two(8 * i + 2), two(8 * i + 4), two(8 * i + 6));
                    }
                }
                const bool seen = settle(l, m, bad);
                if (valid) *reinterpret_cast<float4*>(a.part2_ml + at * 4) = make_float4(seen ? m - kShift : dev::kNegInf, l, back, 0.f);
                fence_before();
            }
        }
    } else if (warp < S::kSoftWarps + kUnpackWarps) {
        // ================= unpacking: warp u takes pair u / 2 of a tile's cells, K (even) or V (odd)
        const int u = warp - S::kSoftWarps, pr = u >> 1;
        const bool is_v = u & 1;
        const int cps = a.g.page_shift - 4, cpp = 1 << cps;
        int tile_no = 0;
        bool ok = true;
        Raw<NBT, F8> raw;
        Scales<NB> scales;
        const uint8_t *c0 = nullptr, *c1 = nullptr;
        int pages[2];                                          // of the tile after next, on their way
        // page numbers of pair pr of tile t of a part; -2: beyond its rows
        auto look_up = [&](const Part& p, int t) {
            const int* table = a.tables + (long long)p.gs * a.g.max_pages;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int C = (p.t0 + t) * (kTileRows / 16) + 2 * pr + i;
                pages[i] = t < p.tb && C * 16 < p.hi ? table[C >> cps] : -2;
            }
        };
        // their cells; nullptr: none, or a bad page
        auto find = [&](const Part& p, int t) {
            const uint8_t* c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int C = (p.t0 + t) * (kTileRows / 16) + 2 * pr + i, pg = pages[i];
                c[i] = nullptr;
                if (pg == -2) continue;
                if (pg < 0 || pg >= a.g.n_pages) {
                    if (lane == 0) atomicExch(a.g.err, kErrCounter);
                    continue;
                }
                c[i] = a.g.pool + pg * a.g.page_bytes + (long long)(p.kh * cpp + (C & (cpp - 1))) * a.g.cell_bytes;
            }
            c0 = c[0];
            c1 = c[1];
        };
        auto fetch = [&](int part) {
            if (is_v) load_v<NB, NBT, F8>(c0, c1, part * NBT, lane, raw);
            else load_k<NB, NBT, F8>(c0, c1, part * NBT, lane, raw);
            if (!F8 && !is_v && part == 0) scales.load(c0, c1, lane);
        };
        for (long long x = xs; x < x1 && ok;) {
            const Part p = part_at(x);
            x += p.tb - p.ta;
            look_up(p, p.ta);
            find(p, p.ta);
            fetch(0);
            look_up(p, p.ta + 1);
            for (int t = p.ta; t < p.tb; ++t, ++tile_no) {
                const int st = tile_no % ST;
                if (tile_no >= ST) {
                    ok = wait(bars.kv_free[st], (uint32_t)(tile_no / ST - 1) & 1u);
                    if (!ok) break;
                }
                const uint32_t tile = kv_tile + (uint32_t)(2 * st + (is_v ? 1 : 0)) * S::tile;
                uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                const int rows = p.hi - ((p.t0 + t) * kTileRows + 32 * pr);      // of the pair that are rows of the prefix
                if (rows < 32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + 2 * (lane & 3);
                        keep[i] = (r < rows ? 0x0000ffffu : 0u) | (r + 1 < rows ? 0xffff0000u : 0u);
                    }
                }
                int shift = 0;
                if (!is_v) {
                    if (!F8) shift = scales.shift(rows, lane);
                    if (lane == 0) s_ok[st][pr] = (c0 || rows <= 0 ? 1 : 0) | (c1 || rows <= 16 ? 2 : 0) | shift << 2;
                }
#pragma unroll 1
                for (int part = 0; part < NQ4; ++part) {
                    if (part > 0) fetch(part);
                    if (is_v) store_v<NB, NBT, F8>(tile, pr, part * NBT, lane, keep, raw);
                    else store_k<NB, NBT, F8>(tile, pr, part * NBT, lane, shift, raw);
                }
                if (t + 1 < p.tb) {
                    find(p, t + 1);
                    fetch(0);                                  // in flight while the products catch up
                    look_up(p, t + 2);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(dev::smem_u32(&bars.kv_full[st]));
            }
        }
    } else if (lane == 0) {
        // ================= products
        constexpr uint32_t idesc_s = instr_desc(128, kTileRows), idesc_o = instr_desc(128, D);
        uint32_t n_part = 0, n_tile[2] = {0, 0};
        int tile_no = 0;
        bool ok = true;
        for (long long x = xs; x < x1 && ok; ++n_part) {
            const Part p = part_at(x);
            x += p.tb - p.ta;
            const int nqt = min(QT, (p.nq - p.qb * QB + 127) / 128);
            ok = wait(bars.q_ready, n_part & 1u);
            if (!ok) break;
            auto scores = [&](int q, int st) {                 // S_q = Q_q K^T
                const uint64_t qd = smem_desc(q_tile + q * S::tile), kd = smem_desc(kv_tile + 2 * st * S::tile);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (uint32_t)((k >> 2) * (kTileRows * 128) + (k & 3) * 32) >> 4;
                    mma_ss(tmem + q * kSCols, qd + off, kd + off, idesc_s, k > 0);
                }
                mma_commit(dev::smem_u32(&bars.s_full[q]));
            };
            auto values = [&](int q, int st, bool first) {     // O_q += P_q V
                const uint64_t vd = smem_desc(kv_tile + (2 * st + 1) * S::tile);
#pragma unroll
                for (int k = 0; k < kTileRows / 16; ++k) {
                    const uint32_t off = (uint32_t)((k >> 2) * (D * 128) + (k & 3) * 32) >> 4;
                    mma_ts(tmem + kOCol + q * D, tmem + q * kSCols + 8 * k, vd + off, idesc_o, !first || k > 0);
                }
                mma_commit(dev::smem_u32(&bars.o_done[q]));
            };
            ok = wait(bars.kv_full[tile_no % ST], (uint32_t)(tile_no / ST) & 1u);
            if (!ok) break;
            fence_after();
            for (int q = 0; q < nqt; ++q) scores(q, tile_no % ST);
            for (int t = p.ta; t < p.tb && ok; ++t, ++tile_no) {
                const int st = tile_no % ST, sn = (tile_no + 1) % ST;
                const bool next = t + 1 < p.tb;
                for (int q = 0; q < nqt; ++q) {
                    ok = wait(bars.p_ready[q], n_tile[q]++ & 1u);
                    if (!ok) break;
                    fence_after();
                    values(q, st, t == p.ta);
                    if (q == nqt - 1) mma_commit(dev::smem_u32(&bars.kv_free[st]));
                    if (next) {
                        if (q == 0) {
                            // (with one stage the next tile follows this one's last product)
                            ok = wait(bars.kv_full[sn], (uint32_t)((tile_no + 1) / ST) & 1u);
                            if (!ok) break;
                            fence_after();
                        }
                        scores(q, sn);
                    }
                }
            }
        }
    }
    __syncthreads();
    if (s_abort) {                                             // a wait ran out: let products in flight end
        const long long t0 = clock64();
        while (clock64() - t0 < (1LL << 28)) __nanosleep(1000);
        __syncthreads();
    }
    if (warp == S::kWarps - 1) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

template <int NB, bool F8>
cudaError_t launch_t(const SplitArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(prefix_kernel<NB, F8>, done, true);
    if (e != cudaSuccess) return e;
    return launch_dependent(prefix_kernel<NB, F8>, dim3((unsigned)a.G), Shape<NB>::kThreads,
                            Shape<NB>::smem + (size_t)(a.n_groups + 1) * sizeof(PlanEntry), s, a);
}

}  // namespace

int prefix_rows_of(int NB) { return NB == 8 ? 128 : 256; }

cudaError_t launch_prefix(const SplitArgs& a, cudaStream_t s) {
    switch (a.g.NB()) {
        case 2: return a.g.fp8 ? launch_t<2, true>(a, s) : launch_t<2, false>(a, s);
        case 4: return a.g.fp8 ? launch_t<4, true>(a, s) : launch_t<4, false>(a, s);
        default: return a.g.fp8 ? launch_t<8, true>(a, s) : launch_t<8, false>(a, s);
    }
}

}  // namespace paged
}  // namespace kvq
