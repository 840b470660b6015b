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
//
// Measured.  Choosing: 131072 rows of 8 KV heads 20 us (4 MB: some 2 us each for the
// load, a digit's counts and their exchange, twice, the masks and the writing), 4608 rows
// 8, 32 sequences of up to 16384 22 (of 16384 each 25).  These have tables as long as the longest sequence; keys
// are held in shared memory for what a table can hold: with tables of 131072 rows 64 sequences of
// 2000 take 23.6 where tables of 2048 take 16.8, and 32 of 16384 33.5 where 24.7.
// Moving: those 32 to 2000 rows each 70 us, for 291 MB
// of sectors read (a row in five stays, in sectors that it shares with others) and 115
// written, 0.86 of the copy rate (91 MB reach memory within the kernel), in place 79; 131072 rows of E4M3 heads of 64 to 16384 18.8,
// in place 29; 4608 to 4096 4.8 and 9.  A cache with page bounds has them renewed behind the
// move, by a warp for each row that a sequence may keep, of which one a page has work: 250 us more for the 32.
#include "kvq_cluster.cuh"
#include "kvq_paged.cuh"

#include <algorithm>

namespace kvq {
namespace paged {
namespace {

// ------------------------------------------------------------ choosing

constexpr int kBits = 11, kBins = 1 << kBits;
constexpr uint32_t kForced = 0xffffffffu;      // key of a row that stays whatever its score (above infinity's)

// a score as an unsigned integer of the same order; a NaN is the lowest, -0 is 0
__device__ __forceinline__ uint32_t ordered(float s) {
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// (sequence, KV head) blockIdx.x / C, rows [s0, s1) of it
template <int kPick>
__global__ void __launch_bounds__(kPick) select_rows_kernel(const __grid_constant__ RowsArgs a) {
    constexpr int kPickWarps = kPick / 32, BPT = kBins / kPick;    // bins of a thread
    static_assert(BPT == 2 || BPT == 4, "a thread reads its bins in one load");
    extern __shared__ __align__(16) uint32_t s_keys[];
    __shared__ __align__(16) uint32_t s_hist[2][kBins];
    __shared__ uint32_t s_range[cluster::kMaxCluster][2];          // of each block's keys, as it says itself
    __shared__ uint32_t s_taken[cluster::kMaxCluster][2];          // its rows above the threshold, and at it
    __shared__ uint32_t s_lo[kPickWarps], s_hi[kPickWarps];
    __shared__ uint32_t s_digit, s_need, s_whole;
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
    cluster::arrive();
    const int first = a.n_first, last = len - a.n_last;           // rows [first, last) compete
    const int per = (((len + C - 1) / C) + 15) & ~15;
    const int s0 = min(len, rank * per), s1 = min(len, s0 + per), m = s1 - s0;
    const int* table = a.tables + (long long)seq * a.g.max_pages;
    const int f0 = min(max(first - s0, 0), m), f1 = min(max(last - s0, f0), m);   // of this part: [f0, f1)
    auto place = [&](int r, int pg) -> const float* {              // of row r's score, in page pg
        if (pg < 0 || pg >= a.g.n_pages) {
            atomicExch(a.g.err, kErrCounter);
            return nullptr;
        }
        return a.scores + ((long long)pg * a.g.Hkv + h) * a.g.page_rows + (r & (a.g.page_rows - 1));
    };
    // ---- keys (four rows a load: they start at a multiple of 16)
    uint32_t lo = 0xffffffffu, hi = 0u;
    const int held = min(m, a.cap);
    const bool all_held = held == m;
    auto keys_of = [&](int i, const float* p, float4 v, uint32_t (&k)[4]) {      // of rows s0 + i .. + 3 from their scores v at p
        k[0] = ordered(v.x); k[1] = ordered(v.y); k[2] = ordered(v.z); k[3] = ordered(v.w);
#pragma unroll
        for (int u = 0; u < 4; ++u) k[u] = i + u >= f0 && i + u < f1 ? (p ? k[u] : 0u) : kForced;
    };
    constexpr int W = 4;                                           // loads in flight, and the next ones' pages
    int pg[W];
    auto pages = [&](int i0) {
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const int i = i0 + 4 * x * kPick;
            pg[x] = i < m ? table[(s0 + i) >> a.g.page_shift] : 0;
        }
    };
    pages(4 * tid);
    for (int i0 = 4 * tid; i0 < m; i0 += 4 * W * kPick) {
        const float* p[W];
        float4 v[W];
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const int i = i0 + 4 * x * kPick;
            p[x] = i < m ? place(s0 + i, pg[x]) : nullptr;
            v[x] = p[x] ? *reinterpret_cast<const float4*>(p[x]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        pages(i0 + 4 * W * kPick);
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const int i = i0 + 4 * x * kPick;
            if (i >= m) break;
            uint32_t k[4];
            keys_of(i, p[x], v[x], k);
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
    cluster::started();
    if (warp < 2) {
        uint32_t v = warp ? 0u : 0xffffffffu;
        if (lane < kPickWarps) v = warp ? s_hi[lane] : s_lo[lane];
        v = warp ? __reduce_max_sync(0xffffffffu, v) : __reduce_min_sync(0xffffffffu, v);
        if (lane < C) cluster::store(cluster::map(&s_range[rank][warp], lane), v);
    }
    cluster::sync();
    lo = s_range[0][0];
    hi = s_range[0][1];
    for (int r = 1; r < C; ++r) {
        lo = min(lo, s_range[r][0]);
        hi = max(hi, s_range[r][1]);
    }
    // keys of rows s0 + i .. + 3, i a multiple of 4 below m (kForced behind the part, too, where they are read again)
    auto four = [&](int i, uint32_t (&k)[4]) {
        if (all_held || i < held) {
            const uint4 v = *reinterpret_cast<const uint4*>(s_keys + i);
            k[0] = v.x; k[1] = v.y; k[2] = v.z; k[3] = v.w;
        } else {
            const float* p = place(s0 + i, table[(s0 + i) >> a.g.page_shift]);
            keys_of(i, p, p ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f), k);
        }
    };
    // ---- the threshold: digit by digit from the top, until all keys that share the digits are wanted
    uint32_t need = (uint32_t)(a.keep - a.n_first - a.n_last), prefix = 0;
    const bool any = need > 0;
    bool whole = false;
    int bits = hi > lo ? 32 - __clz(hi - lo) : 0;
    for (int pass = 0; any && bits > 0 && !whole; ++pass) {
        const int shift = max(0, bits - kBits);
        uint32_t* hist = s_hist[pass & 1];
#pragma unroll
        for (int i = 0; i < BPT; ++i) hist[i * kPick + tid] = 0u;
        __syncthreads();
        const uint32_t mask = bits >= 32 ? 0u : 0xffffffffu << bits, digit = (1u << (bits - shift)) - 1u;
#pragma unroll 2
        for (int i = 4 * tid; i < m; i += 4 * kPick) {
            uint32_t k[4];
            four(i, k);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (k[u] != kForced && ((k[u] - lo) & mask) == prefix) atomicAdd(&hist[((k[u] - lo) >> shift) & digit], 1u);
        }
        cluster::sync();
        // thread t sums its bins, kBins - BPT t - 1 downwards, of all blocks; where the count from the top reaches `need`
        uint32_t c[BPT];
        {
            uint4 v4[cluster::kMaxCluster];
            uint2 v2[cluster::kMaxCluster];
#pragma unroll
            for (int r = 0; r < cluster::kMaxCluster; ++r) {       // (all on their way at once)
                v4[r] = make_uint4(0u, 0u, 0u, 0u);
                v2[r] = make_uint2(0u, 0u);
                if (r < C) {
                    const uint32_t at = cluster::map(&hist[kBins - BPT * tid - BPT], r);
                    if constexpr (BPT == 4) v4[r] = cluster::load4(at);
                    else v2[r] = cluster::load2(at);
                }
            }
#pragma unroll
            for (int i = 0; i < BPT; ++i) c[i] = 0u;
#pragma unroll
            for (int r = 0; r < cluster::kMaxCluster; ++r) {
                if constexpr (BPT == 4) {
                    c[0] += v4[r].w; c[1] += v4[r].z; c[2] += v4[r].y; c[BPT - 1] += v4[r].x;
                } else {
                    c[0] += v2[r].y; c[1] += v2[r].x;
                }
            }
        }
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < BPT; ++i) sum += c[i];
        uint32_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_lo[warp] = x;
        __syncthreads();
        const uint32_t w = lane < warp ? s_lo[lane] : 0u;          // (at most 32 warps)
        uint32_t before = x - sum + __reduce_add_sync(0xffffffffu, w);
        if (before < need && before + sum >= need) {
            int i = 0;
#pragma unroll
            for (int k = 0; k < BPT - 1; ++k)
                if (i == k && before + c[k] < need) {
                    before += c[k];
                    i = k + 1;
                }
            uint32_t in = c[0];
#pragma unroll
            for (int k = 1; k < BPT; ++k)
                if (i == k) in = c[k];
            s_digit = (uint32_t)(kBins - BPT * tid - 1 - i);
            s_need = need - before;
            s_whole = in == need - before;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_need;
        whole = s_whole;
        bits = shift;
    }
    // ---- keys from `from` on are taken, and of those at `at_key` the first `need`, in
    // index order (forced ones have the highest key): a stretch of the part for each
    // warp, 32 rows a step, whose masks lane `step` keeps
    const uint32_t at_key = lo + prefix, from = !any ? kForced : whole ? at_key : at_key + 1u;
    const bool ties = any && !whole;
    constexpr int kGroup = 32 * 32;
    const int stretch = ((m + kPickWarps - 1) / kPickWarps + 31) & ~31;
    const int b0 = min(m, warp * stretch), b1 = min(m, b0 + stretch);
    auto masks = [&](int base, uint32_t& up, uint32_t& same) {     // of rows base + 32 lane .. + 31
        up = same = 0u;
#pragma unroll 8
        for (int st = 0; st < 32; ++st) {
            const int i = base + 32 * st + lane;
            if (base + 32 * st >= b1) break;
            uint32_t k = 0u;
            bool in = i < b1;
            if (in) {
                if (all_held || i < held) {
                    k = s_keys[i];
                } else {
                    const float* p = place(s0 + i, table[(s0 + i) >> a.g.page_shift]);
                    k = i >= f0 && i < f1 ? (p ? ordered(*p) : 0u) : kForced;
                }
            }
            const uint32_t u = __ballot_sync(0xffffffffu, in && k >= from);
            if (lane == st) up = u;
            if (ties) {
                const uint32_t e = __ballot_sync(0xffffffffu, in && k == at_key);
                if (lane == st) same = e;
            }
        }
    };
    uint32_t up0 = 0, same0 = 0, above = 0, equal = 0;             // (of the first group, kept for the writing)
    for (int base = b0; base < b1; base += kGroup) {
        uint32_t up, same;
        masks(base, up, same);
        if (base == b0) {
            up0 = up;
            same0 = same;
        }
        above += __popc(up);
        equal += __popc(same);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    __syncthreads();                                               // (s_lo may still be read)
    if (lane == 0) {
        s_lo[warp] = above;
        s_hi[warp] = equal;
    }
    __syncthreads();
    if (warp < 2) {
        const uint32_t v = __reduce_add_sync(0xffffffffu, lane < kPickWarps ? (warp ? s_hi[lane] : s_lo[lane]) : 0u);
        if (lane < C) cluster::store(cluster::map(&s_taken[rank][warp], lane), v);
    }
    cluster::sync();                                               // (the last: no block touches another's memory behind it)
    uint32_t pos = __reduce_add_sync(0xffffffffu, (lane < rank ? s_taken[lane][0] : 0u) + (lane < warp ? s_lo[lane] : 0u));
    uint32_t eq = __reduce_add_sync(0xffffffffu, (lane < rank ? s_taken[lane][1] : 0u) + (lane < warp ? s_hi[lane] : 0u));
    const uint32_t below = (1u << lane) - 1u;
    for (int base = b0; base < b1; base += kGroup) {
        uint32_t up = up0, same = same0;
        if (base != b0) masks(base, up, same);
        // rows above, and at it, before this lane's 32
        uint32_t pu = __popc(up), pe = __popc(same);
        const uint32_t mu = pu, me = pe;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, pu, o), z = __shfl_up_sync(0xffffffffu, pe, o);
            if (lane >= o) {
                pu += y;
                pe += z;
            }
        }
        const uint32_t all_u = __shfl_sync(0xffffffffu, pu, 31), all_e = __shfl_sync(0xffffffffu, pe, 31);
        pu += pos - mu;
        pe += eq - me;
#pragma unroll 8
        for (int st = 0; st < 32; ++st) {
            if (base + 32 * st >= b1) break;
            const uint32_t u = __shfl_sync(0xffffffffu, up, st), at_u = __shfl_sync(0xffffffffu, pu, st);
            uint32_t at_e = 0, e = 0;
            if (ties) {
                e = __shfl_sync(0xffffffffu, same, st);
                at_e = __shfl_sync(0xffffffffu, pe, st) + __popc(e & below);
            }
            const bool taken = u >> lane & 1u, tied = (e >> lane & 1u) && at_e < need;
            if (taken || tied) out[at_u + __popc(u & below) + min(at_e, need)] = s0 + base + 32 * st + lane;
        }
        pos += all_u;
        eq += all_e;
    }
}

// ------------------------------------------------------------ moving

// Threads of a block.  In place a window is what a cluster's warps hold, and each
// waits for its slowest load and a barrier: large ones where a cluster has SMs to
// itself (131072 rows of 8 heads to 16384: 39 us, large 29; 32 sequences of up to
// 16384 to 2000: 79 and 89).
constexpr int kMove = 256, kMoveLarge = 512;

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
template <int NB, bool F8, bool IN_PLACE, int THREADS>
__global__ void __launch_bounds__(THREADS) compact_kernel(const __grid_constant__ CompactArgs a) {
    constexpr int CELL = NB * (F8 ? 1024 : 928), kMoveWarps = THREADS / 32;
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
                    if (good(now.src) && !(IN_PLACE && now.r == i)) {
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
        if constexpr (IN_PLACE) cluster::sync();                           // all of this window is read
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

template <int kPick>
static cudaError_t launch_select_t(const RowsArgs& a, unsigned grid, int C, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(select_rows_kernel<kPick>, done, false);
    if (e != cudaSuccess) return e;
    return cluster::launch(select_rows_kernel<kPick>, dim3(grid), C, kPick, (size_t)a.cap * 4, s, a);
}

cudaError_t launch_select_rows(RowsArgs a, int num_sms, cudaStream_t s) {
    const long long keys = (long long)a.n_seq * a.g.Hkv, rows = (long long)a.g.max_pages << a.g.page_shift;
    // blocks of a (sequence, KV head): more while SMs are idle and a part keeps 2048 rows
    int C = 1;
    while (C < cluster::kMaxCluster && keys * C * 2 <= 2LL * num_sms && rows > 2048LL * C) C *= 2;
    const long long part = (rows / C + 31) / 16 * 16;
    a.cap = (int)std::min<long long>(part, 40 * 1024);             // 160 KB; rows behind that are read again in each pass
    // large blocks where each has an SM for itself
    return keys * C <= num_sms && part > 2048 ? launch_select_t<1024>(a, (unsigned)(keys * C), C, s)
                                              : launch_select_t<512>(a, (unsigned)(keys * C), C, s);
}

template <int NB, bool F8>
static cudaError_t launch_compact_t(const CompactArgs& a, int C, bool large, cudaStream_t s) {
    const dim3 grid((unsigned)((long long)a.n_seq * a.g.Hkv * a.blocks));
    if (!a.in_place) return cluster::launch(compact_kernel<NB, F8, false, kMove>, grid, C, kMove, 0, s, a);
    return large ? cluster::launch(compact_kernel<NB, F8, true, kMoveLarge>, grid, C, kMoveLarge, 0, s, a)
                 : cluster::launch(compact_kernel<NB, F8, true, kMove>, grid, C, kMove, 0, s, a);
}

cudaError_t launch_compact(CompactArgs a, int num_sms, cudaStream_t s) {
    const long long keys = (long long)a.n_seq * a.g.Hkv;
    const int cells = (a.most + 15) / 16;
    int C = 1;
    bool large = false;
    if (a.in_place) {
        while (C < cluster::kMaxCluster && C * (kMove / 32) < cells && keys * C < 2LL * num_sms) C *= 2;
        large = keys * C <= num_sms;
        a.blocks = C;
    } else {
        // two rounds of what the SMs hold: a block's start is a chain of four loads, of which a
        // warp's later cells wait for the last only
        const int windows = (cells + kMove / 32 - 1) / (kMove / 32);
        a.blocks = (int)std::min<long long>(windows, std::max<long long>(1, 6LL * num_sms / keys));
    }
    switch (a.g.NB()) {
        case 2: return a.g.fp8 ? launch_compact_t<2, true>(a, C, large, s) : launch_compact_t<2, false>(a, C, large, s);
        case 4: return a.g.fp8 ? launch_compact_t<4, true>(a, C, large, s) : launch_compact_t<4, false>(a, C, large, s);
        default: return a.g.fp8 ? launch_compact_t<8, true>(a, C, large, s) : launch_compact_t<8, false>(a, C, large, s);
    }
}

}  // namespace paged
}  // namespace kvq
