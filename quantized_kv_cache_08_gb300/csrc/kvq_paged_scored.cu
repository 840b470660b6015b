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
// A cell's keys lie in the order of the products' operand registers, so a warp
// loads them from global memory straight into its fragments, the next cell's while
// it multiplies this one's: no shared memory, no barriers and no copies to wait for, and as
// many small blocks an SM as registers allow.  Blocks take equal ranges of the
// cells of all (sequence, KV head) pairs.  Queries stay in shared memory in tiles
// (16 of bf16, 8 of f32 in two fp16 parts), and what does not fit is another pass over
// the range's keys, which then come from L2.  A row's score is one lane's alone and its
// gains are added in the tiles' order: the same bits on every run.
#include "kvq_paged.cuh"
#include "kvq_paged_work.cuh"

#include <algorithm>
#include <type_traits>

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
template <int NB>
constexpr int blocks_of() { return NB == 2 ? 5 : NB == 4 ? 4 : 2; }

struct Row {
    float fac, m, w;
    int lo, hi;
};

// What a warp holds of a cell's keys
template <int NB, bool F8>
struct Keys {
    uint4 k[NB / 2][2];
    uint4 d[F8 ? 1 : NB / 2];
    float old;                     // this lane's row's score
    long long at;                  // where the cell's scores lie, -1: no cell
    int row0;
    bool seen;                     // by a query: the keys are loaded
};

template <int NB, bool F8, bool F32Q>
__global__ void __launch_bounds__(kThreads, blocks_of<NB>()) scored_kernel(const __grid_constant__ ScoredArgs a) {
    constexpr int D = NB * 32, QPI = F32Q ? 8 : 16, NQ = QPI / 8;
    constexpr int CELL = NB * (F8 ? 1024 : 928);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ long long s_wsum[kWarps];
    __shared__ int s_ext[4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int QB = a.slices * QPI;
    uint8_t* qs = smem;
    Row* rows = reinterpret_cast<Row*>(smem + (size_t)a.slices * NB * 1024);
    long long* plan = reinterpret_cast<long long*>(smem + (size_t)a.slices * NB * 1024 + (((size_t)QB * sizeof(Row) + 15) & ~(size_t)15));
    wait_for_earlier();
    let_next_start();
    // ---- cells of each sequence: all below its length (with nothing to fade, those that a query sees)
    auto first_row = [&](int len) { return a.window > 0 ? max(0, len - a.T + 1 - a.window) : 0; };
    auto first_cell = [&](int len) { return a.decay == 1.f ? first_row(len) >> 4 : 0; };
    auto cells = [&](int e) {
        const int len = a.lens[e];
        if (len <= 0 || len > (long long)a.g.max_pages << a.g.page_shift) return 0;      // (reported by the decode)
        return ((len + 15) >> 4) - first_cell(len);
    };
    {
        const int per = (a.n_seq + kThreads - 1) / kThreads;
        long long w = 0;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < a.n_seq) {
                plan[e] = w;
                w += cells(e);
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
    // ---- this block's range: a cell for each of its warps at least
    const long long U = plan[a.n_seq] * a.g.Hkv, G = min((long long)gridDim.x, (U + kWarps - 1) / kWarps);
    if (blockIdx.x >= G) return;
    long long x = U * blockIdx.x / G;
    const long long x1 = U * (blockIdx.x + 1) / G;
    float zero[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.f32 %0, 0f00000000;" : "=f"(zero[i]));
    const uint32_t exps = held(0x64646464u);
    const int cps = a.g.page_shift - 4, mask = (1 << cps) - 1;
    while (x < x1) {
        // ---- fragment: cells [ca, cb) of KV head kh of sequence e
        int e = 0;
        {
            int hi = a.n_seq;
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (plan[mid] * a.g.Hkv <= x) e = mid;
                else hi = mid;
            }
        }
        const long long nc = plan[e + 1] - plan[e], in_e = x - plan[e] * a.g.Hkv;
        const int kh = (int)(in_e / nc);
        const int ca = (int)(in_e - kh * nc), cb = (int)min(nc, ca + (x1 - x));
        x += cb - ca;
        const int len = a.lens[e], c0 = first_cell(len), nq = a.hpk * a.T;
        const int* table = a.tables + (long long)e * a.g.max_pages;
        for (int q0 = 0; q0 < nq; q0 += QB) {
            const int n = min(QB, nq - q0), ns = (n + QPI - 1) / QPI;
            // ---- queries [q0, q0 + n) into tiles, as the decode lays them out; one that
            // adds nothing is zeros with weight 0
            __syncthreads();
            if (tid < 4) s_ext[tid] = tid == 0 || tid == 3 ? 0 : 0x7fffffff;      // lo_max, hi_min, lo_min, hi_max
            __syncthreads();
            for (int r = warp; r < ns * QPI; r += kWarps) {
                float v[NB];
                float2 st = make_float2(0.f, 0.f);
                int lo = 0, hi = 0;
                if (r < n) {
                    const int t = (q0 + r) / a.hpk, h = kh * a.hpk + (q0 + r) - t * a.hpk;
                    const long long at = ((long long)e * a.T + t) * a.Hq + h;
                    hi = len - a.T + t + 1;
                    lo = a.window > 0 ? max(0, hi - a.window) : 0;
                    if (hi > lo) st = a.stats[at];
#pragma unroll
                    for (int b = 0; b < NB; ++b) v[b] = load_q(a.q, at * D + 32 * b + lane, a.bf16);
                }
                const bool on = hi > lo && st.y > 0.f && st.x > kNegInf && st.x < kInf;
                uint32_t am = 0u;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (!on) v[b] = 0.f;
                    am = max(am, __float_as_uint(v[b]) & 0x7fffffffu);
                }
                am = __reduce_max_sync(0xffffffffu, am);
                const int ex = am > 0u ? min(max((int)(am >> 23) - 127 - 9, -117), 118) : 0;
                const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
                if (lane == 0) {
                    rows[r] = Row{factor(a.qscale * __uint_as_float((uint32_t)(127 + ex) << 23)), on ? st.x : 0.f, on ? st.y : 0.f, on ? lo : 0, on ? hi : 0};
                    if (on) {
                        atomicMax(&s_ext[0], lo);
                        atomicMin(&s_ext[1], hi);
                        atomicMin(&s_ext[2], lo);
                        atomicMax(&s_ext[3], hi);
                    }
                }
                const int wi = lane & 7, jj = lane >> 3;
                const int reg = ((wi & 3) >> 1) * 2, half = wi & 1, rr = r % QPI;
                uint8_t* tile = qs + (size_t)(r / QPI) * NB * 1024;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float y = v[b] * up;
                    const __half top = __float2half_rn(y);
                    const int at = (2 * b + (wi >> 2)) * 32 + 4 * (rr & 7) + jj;
                    __half* dst = reinterpret_cast<__half*>(tile + at * 16);
                    if (F32Q) {
                        dst[2 * reg + half] = top;
                        dst[2 * (reg + 1) + half] = __float2half_rn(y - __half2float(top));
                    } else {
                        dst[2 * (reg + (rr >> 3)) + half] = top;
                    }
                }
            }
            __syncthreads();
            const int lo_max = s_ext[0], hi_min = s_ext[1], lo_min = s_ext[2], hi_max = s_ext[3];
            const float decay = q0 == 0 ? a.decay : 1.f;
            // ---- its cells, warp by warp; lane (g, j) keeps row 8 (g / 4) + 2 j + g / 2 % 2 of their scores (g even)
            const int my = 8 * (g >> 2) + 2 * j + ((g >> 1) & 1);
            int pages = 0, from = 32;                              // of the warp's next 32 cells, a lane each
            auto fetch = [&](int c, Keys<NB, F8>& y) {
                y.at = -1;
                if (c >= cb) return;
                if (from == 32) {
                    from = 0;
                    const int cc = c + lane * kWarps;
                    pages = cc < cb ? table[(c0 + cc) >> cps] : 0;
                }
                const int pg = __shfl_sync(0xffffffffu, pages, from++);
                if (pg < 0 || pg >= a.g.n_pages) return;           // (reported by the decode)
                const int in = (c0 + c) & mask;
                y.row0 = (c0 + c) * 16;
                y.at = ((long long)pg * a.g.Hkv + kh) * a.g.page_rows + in * 16;
                y.seen = y.row0 < hi_max && y.row0 + 16 > lo_min;
                y.old = 0.f;
                if (!(g & 1) && decay > 0.f) y.old = a.scores[y.at + my];
                if (!y.seen) return;
                const uint8_t* cell = a.g.pool + (long long)pg * a.g.page_bytes + (long long)(kh * (mask + 1) + in) * CELL;
#pragma unroll
                for (int bp = 0; bp < NB / 2; ++bp) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) y.k[bp][t] = __ldg(reinterpret_cast<const uint4*>(cell + bp * 1024 + t * 512 + lane * 16));
                    if constexpr (!F8) y.d[bp] = __ldg(reinterpret_cast<const uint4*>(cell + 512 * NB + (j * NB + 2 * bp) * 8));
                }
            };
            auto take = [&](const Keys<NB, F8>& y) {
                if (y.at < 0) return;
                float gain[2][2] = {{0.f, 0.f}, {0.f, 0.f}};       // rows 2 j + i + 8 t, this lane's queries
                if (y.seen) {
                    const bool edge = y.row0 < lo_max || y.row0 + 16 > hi_min;
#pragma unroll 1
                    for (int s = 0; s < ns; ++s) {
                        const uint8_t* tile = qs + (size_t)s * NB * 1024;
                        float sc[2][2 * NQ], raw[2][4];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
#pragma unroll
                            for (int i = 0; i < 2 * NQ; ++i) sc[t][i] = 0.f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) raw[t][i] = 0.f;
                        }
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const int bp = b / 2, ee = b % 2;
                            const uint4 a0 = *reinterpret_cast<const uint4*>(tile + (2 * b * 32 + lane) * 16);
                            const uint4 a1 = *reinterpret_cast<const uint4*>(tile + ((2 * b + 1) * 32 + lane) * 16);
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                const uint32_t w0 = ee ? y.k[bp][t].z : y.k[bp][t].x, w1 = ee ? y.k[bp][t].w : y.k[bp][t].y;
                                if constexpr (F8) {
                                    mma_f16(raw[t], a0, f8_pair(w0), f8_pair(w0 >> 16));
                                    mma_f16(raw[t], a1, f8_pair(w1), f8_pair(w1 >> 16));
                                } else {
                                    const float2 d = __half22float2(as_h2(ee ? (t ? y.d[bp].w : y.d[bp].z) : (t ? y.d[bp].y : y.d[bp].x)));
                                    float c[4];
                                    mma_f16_new(c, a0, k_pair(w0, 0x4140u, exps), k_pair(w0, 0x4342u, exps), zero);
                                    mma_f16(c, a1, k_pair(w1, 0x4140u, exps), k_pair(w1, 0x4342u, exps));
                                    if constexpr (F32Q) {
                                        c[0] += c[2];
                                        c[1] += c[3];
                                    }
                                    sc[t][0] = fmaf(c[0], d.x, sc[t][0]);
                                    sc[t][1] = fmaf(c[1], d.y, sc[t][1]);
                                    if constexpr (!F32Q) {
                                        sc[t][2] = fmaf(c[2], d.x, sc[t][2]);
                                        sc[t][3] = fmaf(c[3], d.y, sc[t][3]);
                                    }
                                }
                            }
                        }
                        if constexpr (F8) {
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int i = 0; i < 2 * NQ; ++i) sc[t][i] = F32Q ? raw[t][i] + raw[t][2 + i] : raw[t][i];
                        }
#pragma unroll
                        for (int r = 0; r < NQ; ++r) {
                            const Row w = rows[s * QPI + g + 8 * r];
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float v = sc[t][2 * r + i] * w.fac;
                                    if (a.softcap_b > 0.f) v = a.softcap_b * tanhf(a.softcap_a * v);
                                    float p = ex2(v - w.m) * w.w;
                                    const int at = y.row0 + 8 * t + 2 * j + i;
                                    if (edge && (at < w.lo || at >= w.hi)) p = 0.f;
                                    gain[t][i] += p;
                                }
                        }
                    }
                }
                // ---- over the queries (g): each step halves the rows that a lane keeps
                float v0 = g & 4 ? gain[1][0] : gain[0][0], v1 = g & 4 ? gain[1][1] : gain[0][1];
                v0 += __shfl_xor_sync(0xffffffffu, g & 4 ? gain[0][0] : gain[1][0], 16);
                v1 += __shfl_xor_sync(0xffffffffu, g & 4 ? gain[0][1] : gain[1][1], 16);
                float v = g & 2 ? v1 : v0;
                v += __shfl_xor_sync(0xffffffffu, g & 2 ? v0 : v1, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                if (!(g & 1) && y.row0 + my < len) a.scores[y.at + my] = decay > 0.f ? fmaf(decay, y.old, v) : v;
            };
            if constexpr (NB == 8) {                               // (two cells' keys are more registers than there are)
                Keys<NB, F8> y;
                for (int c = ca + warp; c < cb; c += kWarps) {
                    fetch(c, y);
                    take(y);
                }
            } else {
                Keys<NB, F8> y, z;
                fetch(ca + warp, y);
                for (int c = ca + warp; c < cb; c += 2 * kWarps) {
                    fetch(c + kWarps, z);
                    take(y);
                    fetch(c + 2 * kWarps, y);
                    take(z);
                }
            }
        }
    }
}

template <int NB, bool F8, bool F32Q>
cudaError_t launch_t(ScoredArgs a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(scored_kernel<NB, F8, F32Q>, done, false);
    if (e != cudaSuccess) return e;
    constexpr int QPI = F32Q ? 8 : 16;
    // tiles: all queries of a KV head, or what 32 KB hold
    a.slices = std::min((a.hpk * a.T + QPI - 1) / QPI, 32 / NB);
    const size_t smem = (size_t)a.slices * NB * 1024 + (((size_t)a.slices * QPI * sizeof(Row) + 15) & ~(size_t)15) + (size_t)(a.n_seq + 1) * 8;
    return launch_dependent(scored_kernel<NB, F8, F32Q>, dim3((unsigned)(a.sms * blocks_of<NB>())), kThreads, smem, s, a);
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

}  // namespace paged
}  // namespace kvq
