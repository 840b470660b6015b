// The weights that a decode's queries gave to each row, added to the row scores.
//
// Mathematics.  A row's weight for a query is w 2^(s - m) with s its score in log2
// units and (m, w) what the decode left for the query: the reference of its
// softmax and 1 over the sum of its weights, the sink's share taken in.  The
// weights of all queries of a KV head add up to the row's gain, so rows are
// independent of each other: no maximum, no join, one pass over the keys, which are
// the first 34 of a cell's 58 bytes an element block (32 of 64 in E4M3).  The
// scores s are computed as the decode computes them, on the same instructions, so
// that numerators and denominators agree.
//
// A cell's keys lie in the order of the products' operand registers.  The rows
// are M here (16 of them, both halves of a cell in one product) and 8 queries N, the
// other way round than in the decode, for nothing follows that wants the weights
// in another order: half as many products, and a lane's sums are of two rows only.
// Each warp keeps its own ring of bulk copies of keys, two cells a stage, which share
// the queries' fragments and what goes round a stage.  Blocks are small, several an SM, and
// take equal ranges of the cells of all (sequence, KV head) pairs: while one
// changes its queries the others multiply.  Queries stay in shared memory in tiles of 8
// (f32 ones as two fp16 parts), and what does not fit is another pass over
// the range's keys, which then come from L2.  A row's score is one lane's alone and its
// gains are added in the tiles' order: the same bits on every run.
//
// Measured: 64 sequences of 1024 to 16384 rows, 32 query and 8 KV heads of 128, 108 us
// (keys and scores take 102 at the copy rate) behind the decode's 190; one of 512 rows
// 5; the last 8 rows of 4 sequences in a window of 16384, f32, E4M3, 64 query and 8 KV heads
// of 64: 39, bound by the products of 64 queries in two parts (a tile of 8 at a time: 62).
// Keys loaded straight into registers, a cell ahead, took 304 for the first: what
// was loaded ahead spilled, and a spill waits for its load.
//
// Few queries a KV head (gains_kernel): the decode keeps the scores that it works out, 4
// bytes a row and query, and this pass is a sum over them: 71 MB of the batch's, and its
// row scores' 18 in and out, in some 29 us, 25 alone under ncu, two thirds of its issue slots busy; its
// decode 205 us with the scores' stores.
#include "kvq_paged.cuh"
#include "kvq_paged_work.cuh"

#include <algorithm>
#include <type_traits>

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 8;               // queries
constexpr int kPair = 2;               // cells of a stage
constexpr int kFade = 32;              // cells without a query that cost about as much as one with them
// (what a change of key costs a block, in cells: kSetup)
// Blocks an SM, as registers allow: many queries take two tiles of them at a time.  At
// head_dim 256 shared memory holds fewer (3 with one tile of bf16 queries, else 2), and
// the last of the ranges run behind the others: 16 sequences of 16384 rows, 8 KV heads, 32 bf16
// queries 280 us beside a decode of 425, 16 queries 170 beside 225.
template <int NB, bool MANY>
constexpr int blocks_of() { return NB == 8 ? (MANY ? 3 : 4) : MANY ? 4 : 5; }
template <int NB>
constexpr int stages_of() { return 2; }
template <int NB, bool F8>
constexpr int key_bytes() { return NB * (F8 ? 512 : 544); }
template <int NB, bool F32Q>
constexpr int tile_bytes() { return NB * 512 * (F32Q ? 2 : 1); }

struct Row {
    float fac, m, w;                   // a weight is w 2^(fac x product + m)
    int lo, hi, pad[3];
};

// Shared memory: query tiles, their rows, the plan, then each warp's ring
template <int NB, bool F8, bool F32Q>
__host__ __device__ constexpr size_t ring_at(int slices, int n_seq) {
    return ((size_t)slices * (tile_bytes<NB, F32Q>() + kTile * sizeof(Row)) + (size_t)(n_seq + 1) * 8 + 127) / 128 * 128;
}

template <int NB, bool F8, bool F32Q, bool MANY>
__global__ void __launch_bounds__(kThreads, blocks_of<NB, MANY>()) scored_kernel(const __grid_constant__ ScoredArgs a) {
    constexpr int D = NB * 32, STAGES = stages_of<NB>(), KEYS = key_bytes<NB, F8>(), TILE = tile_bytes<NB, F32Q>();
    constexpr int CELL = NB * (F8 ? 1024 : 928), kSetup = MANY ? 16 : 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_wsum[kWarps];
    __shared__ int s_ext[kWarps][4], s_abort;
    __shared__ long long s_at[kWarps][STAGES][kPair];      // where the scores of a stage's cells lie, -1: no cell
    __shared__ __align__(8) uint64_t s_bar[kWarps][STAGES];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int QB = a.slices * kTile;
    uint8_t* qs = smem;
    Row* rows = reinterpret_cast<Row*>(smem + (size_t)a.slices * TILE);
    long long* plan = reinterpret_cast<long long*>(rows + QB);
    uint8_t* ring = smem + ring_at<NB, F8, F32Q>(a.slices, a.n_seq) + (size_t)warp * STAGES * kPair * KEYS;
    const uint32_t ring_u = dev::smem_u32(ring), bar0 = dev::smem_u32(&s_bar[warp][0]);
    if (lane < STAGES) dev::mbar_init(bar0 + 8u * lane, kPair);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    wait_for_earlier();
    let_next_start();
    // ---- work of each sequence and KV head: its setup, the cells that a query sees, and
    // before them (where scores fade) those that none does, kFade a unit
    auto first_row = [&](int len) { return a.window > 0 ? max(0, len - a.T + 1 - a.window) : 0; };
    auto fading = [&](int len) { return a.decay == 1.f ? 0 : ((first_row(len) >> 4) + kFade - 1) / kFade; };
    auto units = [&](int e) {
        const int len = a.lens[e];
        if (len <= 0 || len > (long long)a.g.max_pages << a.g.page_shift) return 0;      // (reported by the decode)
        return kSetup + ((len + 15) >> 4) - (first_row(len) >> 4) + fading(len);
    };
    {
        const int per = (a.n_seq + kThreads - 1) / kThreads;
        long long w = 0;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < a.n_seq) {
                plan[e] = w;
                w += units(e);
            }
        }
        long long wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o) wi += y;
        }
        if (lane == 31) s_wsum[warp] = wi;
        __syncthreads();
        long long base = wi - w;
        for (int i = 0; i < warp; ++i) base += s_wsum[i];
        for (int i = 0; i < per; ++i)
            if (tid * per + i < a.n_seq) plan[tid * per + i] += base;
        if (tid == kThreads - 1) plan[a.n_seq] = base + w;
        __syncthreads();
    }
    // ---- this block's range: a stage for each of its warps at least
    const long long U = plan[a.n_seq] * a.g.Hkv, G = min((long long)gridDim.x, (U + kPair * kWarps - 1) / (kPair * kWarps));
    if (blockIdx.x >= G) return;
    long long x = U * blockIdx.x / G;
    const long long x1 = U * (blockIdx.x + 1) / G;
    float zero[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.f32 %0, 0f00000000;" : "=f"(zero[i]));
    const uint32_t exps = held(0x64646464u), pick = g & 1 ? 0x7632u : 0x5410u;
    const int cps = a.g.page_shift - 4, mask = (1 << cps) - 1;
    const int my = g + 8 * (j & 1);                        // the row of cell j / 2 of a stage whose score is this lane's
    const uint64_t policy = dev::evict_first_policy();
    int st = 0;
    uint32_t phase = 0;
    while (x < x1) {
        // ---- fragment: units [ua, ub) of KV head kh of sequence e, cells [ca, cb) and those that only fade
        int e = 0;
        {
            int hi = a.n_seq;
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (plan[mid] * a.g.Hkv <= x) e = mid;
                else hi = mid;
            }
        }
        const long long in_e = x - plan[e] * a.g.Hkv;
        const int nc = (int)(plan[e + 1] - plan[e]);
        const int kh = in_e < (1LL << 31) ? (int)((unsigned)in_e / (unsigned)nc) : (int)(in_e / nc);
        const int ua = (int)(in_e - (long long)kh * nc), ub = (int)min((long long)nc, ua + (x1 - x));
        x += ub - ua;
        const int len = a.lens[e], nq = a.hpk * a.T;
        const int lo_row = first_row(len);                 // rows before it no query sees
        const int unseen = lo_row >> 4, nf = fading(len);
        const int fa = max(0, ua - kSetup), fb = max(0, ub - kSetup);      // (a key's first units stand for its setup)
        const int ca = unseen + max(0, fa - nf), cb = unseen + max(0, fb - nf);
        const int* table = a.tables + (long long)e * a.g.max_pages;
        // (four rows a thread)
        for (int r = min(unseen, fa * kFade) * 16 + 4 * tid, end = min(unseen, min(fb, nf) * kFade) * 16; r < end; r += 4 * kThreads) {
            const int page = table[r >> a.g.page_shift];
            if (page < 0 || page >= a.g.n_pages) continue;
            float4* p = reinterpret_cast<float4*>(a.scores + ((long long)page * a.g.Hkv + kh) * a.g.page_rows + (r & (a.g.page_rows - 1)));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.decay > 0.f) {
                v = *p;
                v = make_float4(a.decay * v.x, a.decay * v.y, a.decay * v.z, a.decay * v.w);
            }
            *p = v;
        }
        for (int q0 = 0; q0 < nq && ca < cb; q0 += QB) {
            const int n = min(QB, nq - q0), ns = (n + kTile - 1) / kTile;
            const float decay = q0 == 0 ? a.decay : 1.f;
            // ---- the producer side: the warp's cells in order, a lane holding one of the next 32
            int from = 32, pc = ca + kPair * warp, ps = st;
            long long at = -1;                                     // of the lane's cell: its scores, and its keys (NULL: no cell)
            const uint8_t* keys = nullptr;
            auto produce = [&]() {
                if (pc >= cb) return;
                if (from == 32) {
                    from = 0;
                    const int c = pc + (lane & 1) + (lane >> 1) * (kPair * kWarps);
                    at = -1;
                    keys = nullptr;
                    if (c < cb) {
                        const int in = c & mask, page = table[c >> cps];
                        if (page >= 0 && page < a.g.n_pages) {     // (reported by the decode)
                            at = ((long long)page * a.g.Hkv + kh) * a.g.page_rows + in * 16;
                            keys = a.g.pool + (long long)page * a.g.page_bytes + (long long)(kh * (mask + 1) + in) * CELL;
                        }
                    }
                }
                if ((unsigned)(lane - from) < kPair) {
                    const uint32_t bar = bar0 + 8u * ps;
                    s_at[warp][ps][lane - from] = at;
                    if (keys) {
                        dev::mbar_expect_tx(bar, KEYS);
                        asm volatile(
                            "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                            ::"r"(ring_u + (uint32_t)((ps * kPair + lane - from) * KEYS)), "l"(keys), "r"(KEYS), "r"(bar), "l"(policy)
                            : "memory");
                    } else {
                        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
                    }
                }
                from += kPair;
                pc += kPair * kWarps;
                if (++ps == STAGES) ps = 0;
            };
#pragma unroll 1
            for (int i = 0; i < STAGES; ++i) produce();
            // ---- queries [q0, q0 + n) into tiles; one that adds nothing is zeros with weight 0
            __syncthreads();
            // (a warp's next queries are all on their way before it lays the first out)
            constexpr int QA = MANY && NB < 8 ? 4 : 2;
            int ext[4] = {0, 0x7fffffff, 0x7fffffff, 0};           // lo_max, hi_min, lo_min, hi_max
            for (int r0 = warp; r0 < ns * kTile; r0 += QA * kWarps) {
                float v[QA][NB];
                float2 stat[QA];
                int lo[QA], hi[QA];
#pragma unroll
                for (int i = 0; i < QA; ++i) {
                    const int r = r0 + i * kWarps;
                    stat[i] = make_float2(0.f, 0.f);
                    lo[i] = hi[i] = 0;
#pragma unroll
                    for (int b = 0; b < NB; ++b) v[i][b] = 0.f;
                    if (r < n) {
                        const int t = (q0 + r) / a.hpk, h = kh * a.hpk + (q0 + r) - t * a.hpk;
                        const long long at = ((long long)e * a.T + t) * a.Hq + h;
                        hi[i] = len - a.T + t + 1;
                        lo[i] = a.window > 0 ? max(0, hi[i] - a.window) : 0;
                        if (hi[i] > lo[i]) stat[i] = a.stats[at];
#pragma unroll
                        for (int b = 0; b < NB; ++b) v[i][b] = load_q(a.q, at * D + 32 * b + lane, a.bf16);
                    }
                }
#pragma unroll
                for (int i = 0; i < QA; ++i) {
                    const int r = r0 + i * kWarps;
                    if (r >= ns * kTile) break;
                    const bool on = hi[i] > lo[i] && stat[i].y > 0.f && stat[i].x > kNegInf && stat[i].x < kInf;
                    uint32_t am = 0u;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        if (!on) v[i][b] = 0.f;
                        am = max(am, __float_as_uint(v[i][b]) & 0x7fffffffu);
                    }
                    am = __reduce_max_sync(0xffffffffu, am);
                    const int ex = am > 0u ? min(max((int)(am >> 23) - 127 - 9, -117), 118) : 0;
                    const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
                    if (lane == 0) {
                        rows[r] = Row{factor(a.qscale * __uint_as_float((uint32_t)(127 + ex) << 23)), on ? -stat[i].x : 0.f, on ? stat[i].y : 0.f, on ? lo[i] : 0, on ? hi[i] : 0, {}};
                    }
                    if (on) {
                        ext[0] = max(ext[0], lo[i]);
                        ext[1] = min(ext[1], hi[i]);
                        ext[2] = min(ext[2], lo[i]);
                        ext[3] = max(ext[3], hi[i]);
                    }
                    const int wi = lane & 7, jj = lane >> 3;
                    uint8_t* tile = qs + (size_t)(r / kTile) * TILE + (4 * (r % kTile) + jj) * 8 + ((wi & 3) >> 1) * 4 + (wi & 1) * 2;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float y = v[i][b] * up;
                        const __half top = __float2half_rn(y);
                        __half* dst = reinterpret_cast<__half*>(tile + (2 * b + (wi >> 2)) * 256);
                        *dst = top;
                        if constexpr (F32Q) dst[NB * 256] = __float2half_rn(y - __half2float(top));      // the low parts lie behind
                    }
                }
            }
            if (lane < 4) s_ext[warp][lane] = lane == 0 ? ext[0] : lane == 1 ? ext[1] : lane == 2 ? ext[2] : ext[3];
            __syncthreads();
            int lo_max = 0, hi_min = 0x7fffffff, lo_min = 0x7fffffff, hi_max = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                lo_max = max(lo_max, s_ext[w][0]);
                hi_min = min(hi_min, s_ext[w][1]);
                lo_min = min(lo_min, s_ext[w][2]);
                hi_max = max(hi_max, s_ext[w][3]);
            }
            // ---- its cells, warp by warp; the next stage's scores are on their way
            auto old_of = [&](int stage, int c) {
                float v = 0.f;
                if (c < cb && decay > 0.f) {
                    const long long to = s_at[warp][stage][j >> 1];
                    if (to >= 0) v = a.scores[to + my];
                }
                return v;
            };
            __syncwarp();
            float old = old_of(st, ca + kPair * warp);
            for (int c = ca + kPair * warp; c < cb; c += kPair * kWarps) {
                const bool there = wait_bounded(bar0 + 8u * st, phase, &s_abort, a.g.err);
                const int row0 = c * 16;
                const long long to = s_at[warp][st][j >> 1];
                const float next = old_of(st + 1 == STAGES ? 0 : st + 1, c + kPair * kWarps);
                float gain[kPair][2] = {{0.f, 0.f}, {0.f, 0.f}};   // rows g and g + 8 of the cells, this lane's queries
                if (there && row0 < hi_max && row0 + 16 * kPair > lo_min) {
                    // (what the ring holds in the place of a cell that is none reaches no other's sums, and is not stored)
                    const uint8_t* cell = ring + st * kPair * KEYS;
                    const bool edge = row0 < lo_max || row0 + 16 * kPair > hi_min;
                    // products of TB tiles of queries with the stage's cells, and their weights
                    auto tiles = [&](auto tb, int s) {
                        constexpr int TB = decltype(tb)::value;
                        const uint8_t* tile = qs + (size_t)s * TILE + lane * 8;
                        float sc[TB][kPair][4] = {};               // (g, 2 j), (g, 2 j + 1), (g + 8, 2 j), (g + 8, 2 j + 1)
                        [[maybe_unused]] float lows[F8 && F32Q ? TB : 1][kPair][4] = {};
#pragma unroll 1                                           // (unrolled, its loads take more registers than there are)
                        for (int bp = 0; bp < NB / 2; ++bp) {
                            [[maybe_unused]] uint4 k0[kPair], k1[kPair], ks[kPair];      // ks: d of rows 2 (g / 2) + s and + 8, blocks 2 bp and 2 bp + 1
#pragma unroll
                            for (int x = 0; x < kPair; ++x) {
                                k0[x] = *reinterpret_cast<const uint4*>(cell + x * KEYS + bp * 1024 + lane * 16);
                                k1[x] = *reinterpret_cast<const uint4*>(cell + x * KEYS + bp * 1024 + 512 + lane * 16);
                                if constexpr (!F8) ks[x] = *reinterpret_cast<const uint4*>(cell + x * KEYS + 512 * NB + ((g >> 1) * NB + 2 * bp) * 8);
                            }
#pragma unroll
                            for (int ee = 0; ee < 2; ++ee) {
                                const int b = 2 * bp + ee;
                                [[maybe_unused]] uint2 b0[TB], b1[TB], l0[TB], l1[TB];
#pragma unroll
                                for (int u = 0; u < TB; ++u) {
                                    const uint8_t* f = tile + u * TILE + 2 * b * 256;
                                    b0[u] = *reinterpret_cast<const uint2*>(f);
                                    b1[u] = *reinterpret_cast<const uint2*>(f + 256);
                                    if constexpr (F32Q) {
                                        l0[u] = *reinterpret_cast<const uint2*>(f + NB * 512);
                                        l1[u] = *reinterpret_cast<const uint2*>(f + NB * 512 + 256);
                                    }
                                }
#pragma unroll
                                for (int x = 0; x < kPair; ++x) {
                                    const uint32_t v0 = ee ? k0[x].z : k0[x].x, w0 = ee ? k0[x].w : k0[x].y, v1 = ee ? k1[x].z : k1[x].x, w1 = ee ? k1[x].w : k1[x].y;
                                    uint4 p, q;
                                    [[maybe_unused]] float2 d;
                                    if constexpr (F8) {
                                        p = make_uint4(f8_pair(v0), f8_pair(v1), f8_pair(v0 >> 16), f8_pair(v1 >> 16));
                                        q = make_uint4(f8_pair(w0), f8_pair(w1), f8_pair(w0 >> 16), f8_pair(w1 >> 16));
                                    } else {
                                        p = make_uint4(k_pair(v0, 0x4140u, exps), k_pair(v1, 0x4140u, exps), k_pair(v0, 0x4342u, exps), k_pair(v1, 0x4342u, exps));
                                        q = make_uint4(k_pair(w0, 0x4140u, exps), k_pair(w1, 0x4140u, exps), k_pair(w0, 0x4342u, exps), k_pair(w1, 0x4342u, exps));
                                        d = __half22float2(as_h2(__byte_perm(ee ? ks[x].z : ks[x].x, ee ? ks[x].w : ks[x].y, pick)));
                                    }
#pragma unroll
                                    for (int u = 0; u < TB; ++u) {
                                        // (the low parts' sums apart until the end, as the decode has them: the same numbers)
                                        [[maybe_unused]] float acc[4];
                                        if constexpr (F8) {
                                            mma_f16(sc[u][x], p, b0[u].x, b0[u].y);
                                            mma_f16(sc[u][x], q, b1[u].x, b1[u].y);
                                            if constexpr (F32Q) {
                                                mma_f16(lows[u][x], p, l0[u].x, l0[u].y);
                                                mma_f16(lows[u][x], q, l1[u].x, l1[u].y);
                                            }
                                        } else {
                                            mma_f16_new(acc, p, b0[u].x, b0[u].y, zero);
                                            mma_f16(acc, q, b1[u].x, b1[u].y);
                                            if constexpr (F32Q) {
                                                float low[4];
                                                mma_f16_new(low, p, l0[u].x, l0[u].y, zero);
                                                mma_f16(low, q, l1[u].x, l1[u].y);
#pragma unroll
                                                for (int i = 0; i < 4; ++i) acc[i] += low[i];
                                            }
                                        }
                                        if constexpr (!F8) {
                                            sc[u][x][0] = fmaf(acc[0], d.x, sc[u][x][0]);
                                            sc[u][x][1] = fmaf(acc[1], d.x, sc[u][x][1]);
                                            sc[u][x][2] = fmaf(acc[2], d.y, sc[u][x][2]);
                                            sc[u][x][3] = fmaf(acc[3], d.y, sc[u][x][3]);
                                        }
                                    }
                                }
                            }
                        }
                        if constexpr (F8 && F32Q) {
#pragma unroll
                            for (int u = 0; u < TB; ++u)
#pragma unroll
                                for (int x = 0; x < kPair; ++x)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) sc[u][x][i] += lows[u][x][i];
                        }
#pragma unroll
                        for (int u = 0; u < TB; ++u) {
                            const Row* w = rows + (s + u) * kTile + 2 * j;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float4 f = *reinterpret_cast<const float4*>(w + i);      // fac, m, w, lo
#pragma unroll
                                for (int x = 0; x < kPair; ++x)
#pragma unroll
                                    for (int r = 0; r < 2; ++r) {
                                        // (rounded before the reference is taken off, as in the decode: at scores of
                                        // thousands one rounding less would be another number than its sums hold)
                                        float v = __fmul_rn(sc[u][x][2 * r + i], f.x);
                                        if (a.softcap_b > 0.f) v = __fmul_rn(a.softcap_b, tanhf(__fmul_rn(a.softcap_a, v)));
                                        float p = ex2(__fadd_rn(v, f.y));
                                        if (edge) {
                                            const int at_row = row0 + 16 * x + g + 8 * r;
                                            if (at_row < w[i].lo || at_row >= w[i].hi) p = 0.f;
                                        }
                                        gain[x][r] = fmaf(p, f.z, gain[x][r]);
                                    }
                            }
                        }
                    };
                    if constexpr (MANY) {
                        int s = 0;
#pragma unroll 1
                        for (; s + 1 < ns; s += 2) tiles(std::integral_constant<int, 2>{}, s);
                        if (s < ns) tiles(std::integral_constant<int, 1>{}, s);
                    } else {
                        tiles(std::integral_constant<int, 1>{}, 0);
                    }
                }
                // ---- over the queries (j): the first step leaves each lane one of the cells, the second one of its two rows
                const bool up = j & 2, odd = j & 1;
                float v0 = up ? gain[1][0] : gain[0][0], v1 = up ? gain[1][1] : gain[0][1];
                v0 += __shfl_xor_sync(0xffffffffu, up ? gain[0][0] : gain[1][0], 2);
                v1 += __shfl_xor_sync(0xffffffffu, up ? gain[0][1] : gain[1][1], 2);
                float v = odd ? v1 : v0;
                v += __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
                if (to >= 0 && row0 + 16 * (j >> 1) + my < len && there) a.scores[to + my] = decay > 0.f ? fmaf(decay, old, v) : v;
                old = next;
                __syncwarp();                                      // (the stage is read)
                if (there) produce();
                __syncwarp();
                if (++st == STAGES) {
                    st = 0;
                    phase ^= 1u;
                }
            }
        }
    }
    if (s_abort) {                                         // a wait ran out: let copies in flight land before the block ends
        const long long t0 = clock64();
        while (clock64() - t0 < (1LL << 30)) __nanosleep(1000);
    }
}

// ------------------------------------------------------------ from kept scores

constexpr int kGainThreads = 256;
constexpr int kGainSets = 2;           // sets of four rows of a thread in an item

// Rows of (sequence, KV head) pairs, four neighbours a load: their kept scores of NQ
// queries at most, the weights, and the rows' scores.
template <int NQ>
__global__ void __launch_bounds__(kGainThreads) gains_kernel(const __grid_constant__ ScoredArgs a) {
    constexpr int kWarpsG = kGainThreads / 32, kItem = 4 * kGainSets * kGainThreads;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ long long s_sum[kWarpsG];
    long long* plan = reinterpret_cast<long long*>(smem);                      // items before each sequence, of a KV head
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nq = a.hpk * a.T;
    wait_for_earlier();
    let_next_start();
    auto first_row = [&](int len) {                        // (with nothing to fade, rows that a query sees)
        return a.decay == 1.f && a.window > 0 ? max(0, len - a.T + 1 - a.window) & ~15 : 0;
    };
    auto items = [&](int e) {
        const int len = a.lens[e];
        if (len <= 0 || len > (long long)a.g.max_pages << a.g.page_shift) return 0;      // (reported by the decode)
        return (len - first_row(len) + kItem - 1) / kItem;
    };
    {
        const int per = (a.n_seq + kGainThreads - 1) / kGainThreads;
        long long w = 0;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < a.n_seq) {
                plan[e] = w;
                w += items(e);
            }
        }
        long long wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o) wi += y;
        }
        if (lane == 31) s_sum[warp] = wi;
        __syncthreads();
        long long base = wi - w;
        for (int i = 0; i < warp; ++i) base += s_sum[i];
        for (int i = 0; i < per; ++i)
            if (tid * per + i < a.n_seq) plan[tid * per + i] += base;
        if (tid == kGainThreads - 1) plan[a.n_seq] = base + w;
        __syncthreads();
    }
    const long long U = plan[a.n_seq] * a.g.Hkv;
    const int mask = a.g.page_rows - 1;
    for (long long x = blockIdx.x; x < U; x += gridDim.x) {
        int e = 0;
        {
            int hi = a.n_seq;
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (plan[mid] * a.g.Hkv <= x) e = mid;
                else hi = mid;
            }
        }
        const long long in_e = x - plan[e] * a.g.Hkv, n_items = plan[e + 1] - plan[e];
        const int kh = (int)(in_e / n_items), item = (int)(in_e - kh * n_items);
        const int len = a.lens[e], r0 = first_row(len) + item * kItem + 4 * tid;
        const int seen = a.window > 0 ? max(0, len - a.T + 1 - a.window) : 0;      // rows before it no query sees
        const int* table = a.tables + (long long)e * a.g.max_pages;
        long long at[kGainSets];                           // of the rows' scores, -1: none
        float4 old[kGainSets], s[kGainSets][NQ], gain[kGainSets];
#pragma unroll
        for (int i = 0; i < kGainSets; ++i) {
            const int r = r0 + i * 4 * kGainThreads;
            const int page = r < len ? table[r >> a.g.page_shift] : -1;
            at[i] = page >= 0 && page < a.g.n_pages ? ((long long)page * a.g.Hkv + kh) * a.g.page_rows + (r & mask) : -1;
        }
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kGainSets; ++i) {
            const int r = r0 + i * 4 * kGainThreads;
            const bool on = at[i] >= 0;
            old[i] = on && a.decay > 0.f ? *reinterpret_cast<const float4*>(a.scores + at[i]) : none;
            const float* from = a.kept + (at[i] >> 4) * nq * 16 + (r & 15);
#pragma unroll
            for (int q = 0; q < NQ; ++q) s[i][q] = on && q < nq && r + 4 > seen ? __ldcs(reinterpret_cast<const float4*>(from + q * 16)) : none;
            gain[i] = none;
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            if (q >= nq) break;
            const int t = q / a.hpk, h = kh * a.hpk + q - t * a.hpk;
            const int hi = len - a.T + t + 1, lo = a.window > 0 ? max(0, hi - a.window) : 0;
            if (hi <= lo) continue;
            const float2 st = a.stats[((long long)e * a.T + t) * a.Hq + h];
            if (!(st.y > 0.f && st.x > kNegInf && st.x < kInf)) continue;      // (one that is not finite adds nothing)
            auto add = [&](float& g, float score, int r) {
                const float p = ex2(__fadd_rn(score, -st.x)) * st.y;
                g += r >= lo && r < hi ? p : 0.f;
            };
#pragma unroll
            for (int i = 0; i < kGainSets; ++i) {
                const int r = r0 + i * 4 * kGainThreads;
                add(gain[i].x, s[i][q].x, r);
                add(gain[i].y, s[i][q].y, r + 1);
                add(gain[i].z, s[i][q].z, r + 2);
                add(gain[i].w, s[i][q].w, r + 3);
            }
        }
#pragma unroll
        for (int i = 0; i < kGainSets; ++i) {
            if (at[i] < 0) continue;
            const int r = r0 + i * 4 * kGainThreads;
            auto faded = [&](float o, float g) { return a.decay > 0.f ? fmaf(a.decay, o, g) : g; };
            const float v[4] = {faded(old[i].x, gain[i].x), faded(old[i].y, gain[i].y), faded(old[i].z, gain[i].z), faded(old[i].w, gain[i].w)};
            if (r + 4 <= len) {
                *reinterpret_cast<float4*>(a.scores + at[i]) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r + k < len) a.scores[at[i] + k] = v[k];
            }
        }
    }
}

template <int NB, bool F8, bool F32Q, bool MANY>
cudaError_t launch_many(const ScoredArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(scored_kernel<NB, F8, F32Q, MANY>, done, true);
    if (e != cudaSuccess) return e;
    const size_t smem = ring_at<NB, F8, F32Q>(a.slices, a.n_seq) + (size_t)kWarps * stages_of<NB>() * kPair * key_bytes<NB, F8>();
    return launch_dependent(scored_kernel<NB, F8, F32Q, MANY>, dim3((unsigned)(a.sms * blocks_of<NB, MANY>())), kThreads, smem, s, a);
}

template <int NB, bool F8, bool F32Q>
cudaError_t launch_t(ScoredArgs a, cudaStream_t s) {
    // tiles: all queries of a KV head, or what 16 KB hold
    a.slices = std::min((a.hpk * a.T + kTile - 1) / kTile, 16 * 1024 / tile_bytes<NB, F32Q>());
    return a.slices > 1 ? launch_many<NB, F8, F32Q, true>(a, s) : launch_many<NB, F8, F32Q, false>(a, s);
}

template <int NB>
cudaError_t launch_nb(const ScoredArgs& a, cudaStream_t s) {
    if (a.g.fp8) return a.bf16 ? launch_t<NB, true, false>(a, s) : launch_t<NB, true, true>(a, s);
    return a.bf16 ? launch_t<NB, false, false>(a, s) : launch_t<NB, false, true>(a, s);
}

}  // namespace

cudaError_t launch_scored(const ScoredArgs& a, cudaStream_t s) {
    switch (a.g.NB()) {
        case 2: return launch_nb<2>(a, s);
        case 4: return launch_nb<4>(a, s);
        default: return launch_nb<8>(a, s);
    }
}

cudaError_t launch_gains(const ScoredArgs& a, cudaStream_t s) {
    const size_t smem = (size_t)(a.n_seq + 1) * 8;
    const dim3 grid((unsigned)(a.sms * 6));
    const int nq = a.hpk * a.T;
    if (nq <= 1) return launch_dependent(gains_kernel<1>, grid, kGainThreads, smem, s, a);
    if (nq <= 4) return launch_dependent(gains_kernel<4>, grid, kGainThreads, smem, s, a);
    return launch_dependent(gains_kernel<8>, grid, kGainThreads, smem, s, a);
}

}  // namespace paged
}  // namespace kvq
