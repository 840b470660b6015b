// Eviction: choosing the rows of a sequence that stay by their scores, and moving
// them together.
//
// Choosing.  The `keep` best of a sequence's scores, the first and last rows taken
// whatever theirs, ties to the lower index, in index order.  A cluster of blocks
// takes one (sequence, KV head): each reads its part of the scores once into shared
// memory as ordered integers; a radix search for the threshold goes over the bits in
// which they differ, eleven a pass (counts of each block, added up by every block
// from the others' shared memory); then each block writes the rows above the
// threshold, and of those at it the first that are still wanted, behind what the
// blocks before it take.
//
// Moving.  A warp fills a cell of 16 rows.  The bytes of a row lie in its cell at
// places that depend on its row t = 8 h + 2 j + s in the cell, and lane (g, j) holds
// what the four rows of its j have at its places: it loads those pieces (16 bytes
// where the row has them side by side with its neighbour s, else as they come) from
// the four rows' own cells, picks the halves or bytes of their s with one
// byte-permute a word, and stores whole words: nothing passes through shared
// memory, and of a source cell only the sectors that hold wanted rows are read.
// In place a cluster takes one (sequence, KV head), a window of cells at a time:
// rows only move to lower places, so what a later window reads lies behind what
// this one writes, and the only wait is between a window's loads and its stores.
#include "kvq_cluster.cuh"
#include "kvq_paged.cuh"

#include <algorithm>

namespace kvq {
namespace paged {
namespace {

// ------------------------------------------------------------ choosing

constexpr int kPick = 512;             // threads of a block
constexpr int kPickWarps = kPick / 32;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr uint32_t kForced = 0xffffffffu;      // key of a row that stays whatever its score (above infinity's)

// a score as an unsigned integer of the same order; a NaN is the lowest, -0 is 0
__device__ __forceinline__ uint32_t ordered(float s) {
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// (sequence, KV head) blockIdx.x / C, rows [s0, s1) of it
__global__ void __launch_bounds__(kPick) select_rows_kernel(const __grid_constant__ RowsArgs a) {
    extern __shared__ __align__(16) uint32_t s_keys[];
    __shared__ __align__(16) uint32_t s_hist[2][kBins];
    __shared__ uint32_t s_range[cluster::kMaxCluster][2];          // of each block's keys, as it says itself
    __shared__ uint32_t s_taken[cluster::kMaxCluster][2];          // its rows above the threshold, and at it
    __shared__ uint32_t s_lo[kPickWarps], s_hi[kPickWarps], s_sum[kPickWarps];
    __shared__ uint32_t s_digit, s_need;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = cluster::size(), rank = cluster::rank();
    const int key = blockIdx.x / C, seq = key / a.g.Hkv, h = key - seq * a.g.Hkv;
    wait_for_earlier();
    let_next_start();
    int len = a.lens[seq];
    if (len < 0 || len > (long long)a.g.max_pages << a.g.page_shift) {
        if (tid == 0) atomicExch(a.g.err, kErrCounter);
        len = 0;
    }
    int* out = a.rows + (long long)key * a.keep;
    if (len <= a.keep) {                                           // (the same for all blocks of the cluster)
        for (int i = rank * kPick + tid; i < a.keep; i += C * kPick) out[i] = i < len ? i : -1;
        return;
    }
    const int first = a.n_first, last = len - a.n_last;           // rows [first, last) compete
    const int per = (((len + C - 1) / C) + 15) & ~15;
    const int s0 = min(len, rank * per), s1 = min(len, s0 + per), m = s1 - s0;
    const int* table = a.tables + (long long)seq * a.g.max_pages;
    const int f0 = min(max(first - s0, 0), m), f1 = min(max(last - s0, f0), m);   // of this part: [f0, f1)
    auto place = [&](int r) -> const float* {                      // of row r's score
        const int pg = table[r >> a.g.page_shift];
        if (pg < 0 || pg >= a.g.n_pages) {
            atomicExch(a.g.err, kErrCounter);
            return nullptr;
        }
        return a.scores + ((long long)pg * a.g.Hkv + h) * a.g.page_rows + (r & (a.g.page_rows - 1));
    };
    // ---- keys (four rows a load: they start at a multiple of 16)
    uint32_t lo = 0xffffffffu, hi = 0u;
    const int held = min(m, a.cap);
    auto four_of = [&](int i, const float* p, uint32_t (&k)[4]) {  // keys of rows s0 + i .. + 3 from their scores at p
        const float4 v = p ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
        k[0] = ordered(v.x); k[1] = ordered(v.y); k[2] = ordered(v.z); k[3] = ordered(v.w);
#pragma unroll
        for (int u = 0; u < 4; ++u) k[u] = i + u >= f0 && i + u < f1 ? (p ? k[u] : 0u) : kForced;
    };
    for (int i0 = 4 * tid; i0 < m; i0 += 16 * kPick) {
        const float* p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = i0 + 4 * x * kPick < m ? place(s0 + i0 + 4 * x * kPick) : nullptr;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int i = i0 + 4 * x * kPick;
            if (i >= m) break;
            uint32_t k[4];
            four_of(i, p[x], k);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (k[u] != kForced) {
                    lo = min(lo, k[u]);
                    hi = max(hi, k[u]);
                }
            if (i < held) *reinterpret_cast<uint4*>(s_keys + i) = make_uint4(k[0], k[1], k[2], k[3]);   // (cap is a multiple of 4)
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        s_lo[warp] = lo;
        s_hi[warp] = hi;
    }
    __syncthreads();
    if (tid < 2 * C) {
        uint32_t v = tid & 1 ? s_hi[0] : s_lo[0];
        for (int w = 1; w < kPickWarps; ++w) v = tid & 1 ? max(v, s_hi[w]) : min(v, s_lo[w]);
        cluster::store(cluster::map(&s_range[rank][tid & 1], tid >> 1), v);
    }
    cluster::sync();
    lo = s_range[0][0];
    hi = s_range[0][1];
    for (int r = 1; r < C; ++r) {
        lo = min(lo, s_range[r][0]);
        hi = max(hi, s_range[r][1]);
    }
    auto key_of = [&](int i) -> uint32_t {                         // of row s0 + i
        if (i < held) return s_keys[i];
        const float* p = place(s0 + i);
        return p ? ordered(*p) : 0u;
    };
    // ---- the threshold: digit by digit from the top
    uint32_t need = (uint32_t)(a.keep - a.n_first - a.n_last), prefix = 0;
    const bool any = need > 0;
    int bits = hi > lo ? 32 - __clz(hi - lo) : 0;
    for (int pass = 0; any && bits > 0; ++pass) {
        const int shift = max(0, bits - kBits);
        uint32_t* hist = s_hist[pass & 1];
        reinterpret_cast<uint4*>(hist)[tid] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        const uint32_t mask = bits >= 32 ? 0u : 0xffffffffu << bits, digit = (1u << (bits - shift)) - 1u;
#pragma unroll 4
        for (int i = f0 + tid; i < f1; i += kPick) {
            const uint32_t k = key_of(i) - lo;
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
        }
        cluster::sync();
        // thread t sums bins kBins - 4 t - 1 .. - 4 of all blocks; where the count from the top reaches `need`
        uint4 all[cluster::kMaxCluster], c = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int r = 0; r < cluster::kMaxCluster; ++r) {           // (all on their way at once)
            all[r] = make_uint4(0u, 0u, 0u, 0u);
            if (r < C) all[r] = cluster::load4(cluster::map(&hist[kBins - 4 * tid - 4], r));
        }
#pragma unroll
        for (int r = 0; r < cluster::kMaxCluster; ++r) {
            c.x += all[r].x; c.y += all[r].y; c.z += all[r].z; c.w += all[r].w;
        }
        const uint32_t sum = c.x + c.y + c.z + c.w;
        uint32_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_sum[warp] = x;
        __syncthreads();
        uint32_t before = x - sum;
        for (int w = 0; w < warp; ++w) before += s_sum[w];
        if (before < need && before + sum >= need) {
            const uint32_t n[4] = {c.w, c.z, c.y, c.x};
            int i = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (i == k && before + n[k] < need) {
                    before += n[k];
                    i = k + 1;
                }
            s_digit = (uint32_t)(kBins - 4 * tid - 1 - i);
            s_need = need - before;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_need;
        bits = shift;
    }
    const uint32_t thr = any ? lo + prefix : kForced - 1u;         // (no score's key)
    // ---- rows above the threshold, and the first `need` at it, in index order: a
    // stretch of the part for each warp, four neighbours a lane, the counts of 128 in the halves of a word
    const int stretch = ((m + kPickWarps - 1) / kPickWarps + 127) & ~127, b0 = min(m, warp * stretch), b1 = min(m, b0 + stretch);
    auto look = [&](int i, uint32_t& up, uint32_t& same) {         // masks of rows i .. i + 3
        up = same = 0u;
        if (i >= b1) return;
        uint32_t k[4];
        if (i < held) {
            const uint4 v = *reinterpret_cast<const uint4*>(s_keys + i);
            k[0] = v.x; k[1] = v.y; k[2] = v.z; k[3] = v.w;
        } else {
            four_of(i, place(s0 + i), k);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool in = i + u < b1;
            up |= in && k[u] > thr ? 1u << u : 0u;
            same |= in && k[u] == thr ? 1u << u : 0u;
        }
    };
    uint32_t above = 0, at = 0;
#pragma unroll 2
    for (int i = b0 + 4 * lane; i < b1; i += 128) {
        uint32_t up, same;
        look(i, up, same);
        above += __popc(up);
        at += __popc(same);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    at = __reduce_add_sync(0xffffffffu, at);
    if (lane == 0) {
        s_lo[warp] = above;
        s_hi[warp] = at;
    }
    __syncthreads();
    if (tid < 2 * C) {
        uint32_t v = 0;
        for (int w = 0; w < kPickWarps; ++w) v += tid & 1 ? s_hi[w] : s_lo[w];
        cluster::store(cluster::map(&s_taken[rank][tid & 1], tid >> 1), v);
    }
    cluster::sync();                                               // (the last: no block touches another's memory behind it)
    uint32_t pos = 0, eq = 0;
    for (int r = 0; r < rank; ++r) {
        pos += s_taken[r][0];
        eq += s_taken[r][1];
    }
    for (int w = 0; w < warp; ++w) {
        pos += s_lo[w];
        eq += s_hi[w];
    }
    for (int i0 = b0; i0 < b1; i0 += 128) {
        uint32_t up, same;
        look(i0 + 4 * lane, up, same);
        const uint32_t mine = __popc(up) | __popc(same) << 16;
        uint32_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, sum, 31), before = sum - mine;
        uint32_t to = pos + (before & 0xffffu), e = eq + (before >> 16);      // rows above, and at it, before this lane's
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (up >> u & 1u) out[to++ + min(e, need)] = s0 + i0 + 4 * lane + u;
            if (same >> u & 1u) {
                if (e < need) out[to + e] = s0 + i0 + 4 * lane + u;
                ++e;
            }
        }
        pos += all & 0xffffu;
        eq += all >> 16;
    }
}

// ------------------------------------------------------------ moving

constexpr int kMove = 256;             // threads of a block
constexpr int kMoveWarps = kMove / 32;

template <typename T>
__device__ __forceinline__ T get(const uint8_t* p) { return *reinterpret_cast<const T*>(p); }

// words of two neighbouring rows (s = 0, 1) from the words that hold them: their
// half words (16-bit pieces) or every other byte, of the rows' own s
__device__ __forceinline__ uint32_t halves(uint32_t sa, uint32_t sb) { return (sa ? 0x0032u : 0x0010u) | (sb ? 0x7600u : 0x5400u); }
__device__ __forceinline__ uint32_t bytes_of(uint32_t sa, uint32_t sb) {
    return sa | (4u + sb) << 4 | (sa + 2u) << 8 | (6u + sb) << 12;
}
__device__ __forceinline__ uint4 blend(const uint4& x, const uint4& y, uint32_t sel) {
    return make_uint4(__byte_perm(x.x, y.x, sel), __byte_perm(x.y, y.y, sel), __byte_perm(x.z, y.z, sel), __byte_perm(x.w, y.w, sel));
}

// What lane (g, j) holds of a cell: its pieces of rows t = 8 h + 2 j + s, index 2 h + s
template <int NB, bool F8>
struct Piece {
    static constexpr int KC = NB == 8 ? 2 : 1, KR = NB == 2 ? 2 : 4;          // key chunks of 16 bytes a row, rows
    static constexpr int VR = F8 ? NB : NB == 8 ? 4 : NB == 4 ? 2 : 1;        // 512-byte regions of V
    uint4 k[KC][KR];
    uint4 v[VR];
    uint32_t nib[F8 ? 1 : VR];
    uint2 kd;
    uint4 dm;

    // from the cells of the four rows and their rows in them
    __device__ __forceinline__ void load(const uint8_t* const (&cell)[4], const int (&t)[4], int g, int j) {
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int r = 0; r < KR; ++r) {
                const int chunk = NB == 2 ? g & 3 : g + 8 * c;
                const uint8_t* from = NB == 2 ? (g >> 2 ? cell[2 + r] : cell[r]) : cell[r];
                const int row = NB == 2 ? (g >> 2 ? t[2 + r] : t[r]) : t[r];
                k[c][r] = get<uint4>(from + (chunk >> 2) * 1024 + row * 64 + (chunk & 3) * 16);
            }
        int hs[4], s[4], lane[4];                         // of the rows where they are: half, s, lane
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hs[i] = t[i] >> 3;
            s[i] = t[i] & 1;
            lane[i] = 4 * g + ((t[i] >> 1) & 3);
        }
        if constexpr (F8) {
            constexpr int RH = NB / 2;                    // regions of a half
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < RH; ++c) {
                    const int x = 2 * h, y = x + 1;
                    const uint4 p = get<uint4>(cell[x] + 512 * NB + (hs[x] * RH + c) * 512 + lane[x] * 16);
                    const uint4 q = get<uint4>(cell[y] + 512 * NB + (hs[y] * RH + c) * 512 + lane[y] * 16);
                    v[h * RH + c] = blend(p, q, bytes_of(s[x], s[y]));
                }
        } else {
            if constexpr (NB == 2) {                      // a lane's 16 bytes hold both halves
                uint32_t w[4], n = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = 2 * h, y = x + 1;
                    const uint2 p = get<uint2>(cell[x] + 544 * NB + lane[x] * 16 + hs[x] * 8), q = get<uint2>(cell[y] + 544 * NB + lane[y] * 16 + hs[y] * 8);
                    const uint32_t sel = halves(s[x], s[y]);
                    w[2 * h] = __byte_perm(p.x, q.x, sel);
                    w[2 * h + 1] = __byte_perm(p.y, q.y, sel);
#pragma unroll
                    for (int i = x; i <= y; ++i)
                        n |= (uint32_t)cell[i][800 * NB + lane[i] * 4 + s[i] * 2 + hs[i]] << (8 * (2 * (i & 1) + h));
                }
                v[0] = make_uint4(w[0], w[1], w[2], w[3]);
                nib[0] = n;
            } else {
                constexpr int RH = NB / 4;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < RH; ++c) {
                        const int x = 2 * h, y = x + 1;
                        const uint32_t sel = halves(s[x], s[y]);
                        const int rx = hs[x] * RH + c, ry = hs[y] * RH + c;
                        v[h * RH + c] = blend(get<uint4>(cell[x] + 544 * NB + rx * 512 + lane[x] * 16), get<uint4>(cell[y] + 544 * NB + ry * 512 + lane[y] * 16), sel);
                        nib[h * RH + c] = __byte_perm(get<uint32_t>(cell[x] + 800 * NB + rx * 128 + lane[x] * 4), get<uint32_t>(cell[y] + 800 * NB + ry * 128 + lane[y] * 4), sel);
                    }
            }
            if (g < NB) {                                 // scales of block g
                uint32_t d[4], e[4], f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int jj = (t[i] >> 1) & 3, four = 2 * hs[i] + s[i];
                    d[i] = get<uint16_t>(cell[i] + 512 * NB + (jj * NB + g) * 8 + four * 2);
                    const uint8_t* at = cell[i] + 864 * NB + (jj * NB + g) * 16 + four * 2;
                    e[i] = get<uint16_t>(at);
                    f[i] = get<uint16_t>(at + 8);
                }
                kd = make_uint2(d[0] | d[1] << 16, d[2] | d[3] << 16);
                dm = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, f[0] | f[1] << 16, f[2] | f[3] << 16);
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t* cell, int g, int j) const {
        const int lane = 4 * g + j;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int r = 0; r < KR; ++r) {
                const int chunk = NB == 2 ? g & 3 : g + 8 * c, i = NB == 2 ? 2 * (g >> 2) + r : r;
                *reinterpret_cast<uint4*>(cell + (chunk >> 2) * 1024 + (8 * (i >> 1) + 2 * j + (i & 1)) * 64 + (chunk & 3) * 16) = k[c][r];
            }
#pragma unroll
        for (int c = 0; c < VR; ++c) {
            *reinterpret_cast<uint4*>(cell + (F8 ? 512 : 544) * NB + c * 512 + lane * 16) = v[c];
            if constexpr (!F8) *reinterpret_cast<uint32_t*>(cell + 800 * NB + c * 128 + lane * 4) = nib[c];
        }
        if (!F8 && g < NB) {
            *reinterpret_cast<uint2*>(cell + 512 * NB + (j * NB + g) * 8) = kd;
            *reinterpret_cast<uint4*>(cell + 864 * NB + (j * NB + g) * 16) = dm;
        }
    }
};

// (sequence, KV head) blockIdx.x / a.blocks, whose blocks take window after window of
// blocks x warps cells; in place they are a cluster.
template <int NB, bool F8>
__global__ void __launch_bounds__(kMove) compact_kernel(const __grid_constant__ CompactArgs a) {
    constexpr int CELL = NB * (F8 ? 1024 : 928);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int key = blockIdx.x / a.blocks, part = blockIdx.x - key * a.blocks;
    const int seq = key / a.g.Hkv, h = key - seq * a.g.Hkv;
    wait_for_earlier();
    let_next_start();
    const int len = a.lens[seq];
    __syncthreads();                                               // (lens_out may be lens: read before this block is counted)
    const bool ok = len >= 0 && len <= (long long)a.g.max_pages << a.g.page_shift;
    if (!ok && tid == 0) atomicExch(a.g.err, kErrCounter);
    const int n = ok ? min(len, a.keep) : 0, cells = (n + 15) >> 4;
    const int* list = a.rows + (long long)key * a.keep;
    const int* from = a.tables + (long long)seq * a.g.max_pages;
    const int* to = a.tables_out + (long long)seq * a.g.max_pages;
    const int cps = a.g.page_shift - 4, mask = (1 << cps) - 1;
    auto good = [&](int page) {
        if (page >= 0 && page < a.g.n_pages) return true;
        atomicExch(a.g.err, kErrCounter);
        return false;
    };
    // What a cell's turn needs is asked for ahead: two turns the list's entries (lane l
    // entry l - 1 of the cell's, lane 0 the one before them), one turn the pages
    const int step = a.blocks * kMoveWarps, first = part * kMoveWarps;
    auto entry = [&](int c) {
        const int i = 16 * c + lane - 1;
        return c < cells && lane <= 16 && i >= 0 && i < n ? list[i] : -1;
    };
    struct Pages {
        int r, prev, src, dst;                                     // of lane < 16: its row, the one before it in the list, pages
    };
    auto pages_of = [&](int c, int e) {
        Pages p{-1, e, -1, -1};
        p.r = __shfl_down_sync(0xffffffffu, e, 1);
        if (c < cells) {
            p.dst = to[(16 * c) >> a.g.page_shift];
            if (lane < 16 && p.r >= 0 && p.r < len) p.src = from[p.r >> a.g.page_shift];
        }
        return p;
    };
    int c = first + warp;
    Pages now = pages_of(c, entry(c));
    int ahead = entry(c + step);
    for (int c0 = first; c0 - first < cells; c0 += step, c += step) {
        const Pages next = pages_of(c + step, ahead);
        ahead = entry(c + 2 * step);
        uint8_t* dst = nullptr;
        long long row_at = 0, score_from = 0, score_to = 0;        // lane t < 16: byte of its row's cell; scores
        int t = lane & 15;
        bool moved = false;
        Piece<NB, F8> p;
        if (c < cells && good(now.dst)) {
            const long long cell = (long long)now.dst * a.g.page_bytes + (long long)(h * (mask + 1) + (c & mask)) * CELL;
            score_to = ((long long)now.dst * a.g.Hkv + h) * a.g.page_rows + (c & mask) * 16 + (lane & 15);
            row_at = cell;                                         // (a row that is not moved stays as it is)
            const int i = 16 * c + lane;
            if (lane < 16 && i < n) {
                if (now.r >= i && now.r > now.prev && now.r < len) {
                    if (good(now.src) && !(a.in_place && now.r == i)) {
                        row_at = (long long)now.src * a.g.page_bytes + (long long)(h * (mask + 1) + ((now.r >> 4) & mask)) * CELL;
                        score_from = ((long long)now.src * a.g.Hkv + h) * a.g.page_rows + (now.r & (a.g.page_rows - 1));
                        t = now.r & 15;
                        moved = true;
                    }
                } else {
                    atomicExch(a.g.err, kErrCounter);
                }
            }
            if (__any_sync(0xffffffffu, moved)) dst = a.g.pool + cell;
        }
        float score = 0.f;
        if (dst) {
            const uint8_t* cell[4];
            int rt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 8 * (i >> 1) + 2 * j + (i & 1);
                cell[i] = a.g.pool + __shfl_sync(0xffffffffu, row_at, at);
                rt[i] = __shfl_sync(0xffffffffu, t, at);
            }
            p.load(cell, rt, g, j);
            if (a.scores && moved) score = a.scores[score_from];
        }
        if (a.in_place) cluster::sync();                           // all of this window is read
        if (dst) {
            p.store(dst, g, j);
            if (a.scores && moved) a.scores[score_to] = score;
        }
        now = next;
    }
    if (tid == 0 && a.lens_out) {
        // the sequence's last block sets the length, when all have read it
        __threadfence();
        const int total = a.blocks * a.g.Hkv;
        if (atomicAdd(a.arrived + seq, 1) == total - 1) {
            a.arrived[seq] = 0;
            a.lens_out[seq] = ok ? n : len;
        }
    }
}

}  // namespace

cudaError_t launch_select_rows(RowsArgs a, int num_sms, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(select_rows_kernel, done, false);
    if (e != cudaSuccess) return e;
    const long long keys = (long long)a.n_seq * a.g.Hkv, rows = (long long)a.g.max_pages << a.g.page_shift;
    // blocks of a (sequence, KV head): more while SMs are idle and a part keeps 2048 rows
    int C = 1;
    while (C < cluster::kMaxCluster && keys * C * 2 <= 2LL * num_sms && rows > 2048LL * C) C *= 2;
    const long long part = (rows / C + 31) / 16 * 16;
    a.cap = (int)std::min<long long>(part, 40 * 1024);             // 160 KB; rows behind that are read again in each pass
    return cluster::launch(select_rows_kernel, dim3((unsigned)(keys * C)), C, kPick, (size_t)a.cap * 4, s, a);
}

template <int NB>
static cudaError_t launch_compact_nb(const CompactArgs& a, int C, cudaStream_t s) {
    const dim3 grid((unsigned)((long long)a.n_seq * a.g.Hkv * a.blocks));
    return a.g.fp8 ? cluster::launch(compact_kernel<NB, true>, grid, C, kMove, 0, s, a)
                   : cluster::launch(compact_kernel<NB, false>, grid, C, kMove, 0, s, a);
}

cudaError_t launch_compact(CompactArgs a, int num_sms, cudaStream_t s) {
    const int windows = ((a.most + 15) / 16 + kMoveWarps - 1) / kMoveWarps;      // blocks that take a cell a warp each
    int C = 1;
    if (a.in_place) {
        while (C < cluster::kMaxCluster && C < windows && (long long)a.n_seq * a.g.Hkv * C < 2LL * num_sms) C *= 2;
        a.blocks = C;
    } else {
        // two rounds of what the SMs hold: a block's start is a chain of four loads, of which a
        // warp's later cells wait for the last only
        a.blocks = (int)std::min<long long>(windows, std::max<long long>(1, 6LL * num_sms / ((long long)a.n_seq * a.g.Hkv)));
    }
    switch (a.g.NB()) {
        case 2: return launch_compact_nb<2>(a, C, s);
        case 4: return launch_compact_nb<4>(a, C, s);
        default: return launch_compact_nb<8>(a, C, s);
    }
}

}  // namespace paged
}  // namespace kvq
