// Choosing the pages that a query reads, by the key bounds of the pages.
//
// A page's score is an upper bound of the query's product with every key in it:
// sum over elements of max(c min, c max) for the query code c, which is c max
// where c > 0 and c min elsewhere, so two integer dot products of the query's
// positive and negative parts give it exactly; the two scales and the sum over
// blocks are single f32 operations in a fixed order.  Scores are therefore the
// same numbers on every run, and ties (common between codes) go to the lowest
// index.  One kernel: a CTA scores 256 pages of a KV head (NB lanes a page), and the last CTA of an (entry, KV
// head) picks: a radix search for the threshold over the bits in which the scores
// differ, eight a pass, until the few that share its digits can be ranked one a
// thread, then a compaction in index order.  131072 rows in pages of 32, 64 query
// and 8 KV heads of 64: 12 us (4.5 MB of bounds are 0.7), bound by the chain from
// the scores through the counter to the pick.
#include "kvq_paged.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPages = 256;            // pages of a CTA
constexpr int kKeep = 8192;            // keys that the pick holds in shared memory
constexpr int kRank = 256;             // keys that are ranked one a thread
constexpr int kBlock = 20;             // words of a query block's codes and scale

// number of pages with a row that query row t sees, 0 for a bad length
__device__ __forceinline__ int page_count(const SelectArgs& a, int seq, int t, bool report) {
    const int len = a.lens[seq];
    if (len < 0 || len > (long long)a.g.max_pages << a.g.page_shift) {
        if (report) atomicExch(a.g.err, kErrCounter);
        return 0;
    }
    const int hi = len - a.T + t + 1;
    return hi > 0 ? (hi + a.g.page_rows - 1) >> a.g.page_shift : 0;
}

// f32 -> an unsigned integer of the same order (-0 counts as 0)
__device__ __forceinline__ uint32_t ordered(float s) {
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The `keep` pages of one (entry, KV head) of np > keep: the first n_first, the
// last n_last and the best keys of the others, ties to the lowest index.
__device__ __forceinline__ void pick(const SelectArgs& a, const uint32_t* g_keys, uint32_t* s_keys, int np, int* out) {
    __shared__ int s_hist[256];
    __shared__ int s_gt[kWarps], s_eq[kWarps];
    __shared__ uint32_t s_lo[kWarps], s_hi[kWarps];
    __shared__ uint32_t s_digit, s_thr, s_key[kRank];
    __shared__ int s_need, s_in, s_count, s_cut, s_idx[kRank];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool in_smem = np <= kKeep;
    const int first = a.n_first, last = np - a.n_last;      // pages [first, last) compete
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 4
    for (int i = 4 * tid; i < np; i += 4 * kThreads) {      // (rows of keys are padded to four)
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(g_keys + i));
        if (in_smem) *reinterpret_cast<uint4*>(s_keys + i) = v;
        const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u >= first && i + u < last) {
                lo = min(lo, k[u]);
                hi = max(hi, k[u]);
            }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        s_lo[warp] = lo;
        s_hi[warp] = hi;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        lo = min(lo, s_lo[w]);
        hi = max(hi, s_hi[w]);
    }
    const uint32_t* keys = in_smem ? s_keys : g_keys;       // (written before the fence that the caller passed)
    auto key = [&](int i) { return keys[i] - lo; };
    // f(index, key) of the competing pages, four neighbours a thread
    auto each = [&](auto f) {
#pragma unroll 2
        for (int i = 4 * tid; i < last; i += 4 * kThreads) {
            const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
            const uint32_t k[4] = {v.x - lo, v.y - lo, v.z - lo, v.w - lo};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u >= first && i + u < last) f(i + u, k[u]);
        }
    };
    int need = a.keep - a.n_first - a.n_last;               // of the competing pages
    uint32_t prefix = 0;
    int bits = hi > lo ? 32 - __clz(hi - lo) : 0;           // in which the keys differ
    int cut = np;                                           // of the keys that equal the threshold, those below this index
    while (bits > 0 && need > 0) {
        const int shift = max(0, bits - 8);
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        const uint32_t mask = bits >= 32 ? 0u : 0xffffffffu << bits;
        each([&](int, uint32_t k) {
            if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << (bits - shift)) - 1u)], 1);
        });
        __syncthreads();
        if (warp == 0) {
            // lane l sums bins 255 - 8 l .. 248 - 8 l; the bin in which the count reaches `need`
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = s_hist[255 - 8 * lane - i];
                sum += c[i];
            }
            int x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            int before = x - sum;
            if (before < need && x >= need) {
                int i = 0;
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (i == k && before + c[k] < need) {
                        before += c[k];
                        i = k + 1;
                    }
                s_digit = (uint32_t)(255 - 8 * lane - i);
                s_need = need - before;
                s_in = c[0];
#pragma unroll
                for (int k = 1; k < 8; ++k)
                    if (i == k) s_in = c[k];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_need;
        bits = shift;
        if (s_in <= kRank && bits > 0) {
            // few keys share the digits: each thread ranks one of them
            if (tid == 0) s_count = 0;
            __syncthreads();
            const uint32_t m = 0xffffffffu << bits;
            each([&](int i, uint32_t k) {
                if ((k & m) == prefix) {
                    const int at = atomicAdd(&s_count, 1);
                    s_key[at] = k;
                    s_idx[at] = i;
                }
            });
            __syncthreads();
            const int n = s_count;
            if (tid < n) {
                const uint32_t k = s_key[tid];
                const int i = s_idx[tid];
                int rank = 0;
#pragma unroll 8
                for (int o = 0; o < n; ++o) rank += s_key[o] > k || (s_key[o] == k && s_idx[o] < i);
                if (rank == need - 1) {                     // the last that is taken
                    s_thr = k;
                    s_cut = i + 1;
                }
            }
            __syncthreads();
            prefix = s_thr;
            cut = s_cut;
            need = np;                                      // (the index decides among equals)
            break;
        }
    }
    // competing keys above the threshold and the first `need` that equal it, in
    // index order: each warp counts its share of the pages, then writes it
    const int per = ((np + kWarps - 1) / kWarps + 31) & ~31, b0 = warp * per, b1 = min(np, b0 + per);
    const bool none = a.keep == a.n_first + a.n_last;
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int base = b0; base < b1; base += 32) {
        const int i = base + lane;
        const bool in = i < b1, forced = in && (i < first || i >= last);
        const uint32_t k = in ? key(i) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, forced || (in && !none && k > prefix)));
        eq += __popc(__ballot_sync(0xffffffffu, in && !forced && !none && k == prefix && i < cut));
    }
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    int at = 0, e0 = 0;
    for (int w = 0; w < warp; ++w) {
        at += s_gt[w];
        e0 += s_eq[w];
    }
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int base = b0; base < b1; base += 32) {
        const int i = base + lane;
        const bool in = i < b1, forced = in && (i < first || i >= last);
        const uint32_t k = in ? key(i) : 0u;
        const bool up = forced || (in && !none && k > prefix), same = in && !forced && !none && k == prefix && i < cut;
        const unsigned mg = __ballot_sync(0xffffffffu, up), me = __ballot_sync(0xffffffffu, same);
        const int rank = e0 + __popc(me & below);           // equal keys before this one
        if (up || (same && rank < need)) out[at + __popc(mg & below) + min(rank, need)] = i;
        at += __popc(mg);
        e0 += __popc(me);
    }
}

// Scores of pages [kPages blockIdx.x, + kPages) for KV head blockIdx.y and entry
// blockIdx.z: NB lanes a page, one 32-element block each; then the pick.
template <int NB>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a) {
    constexpr int D = NB * 32;
    constexpr int PW = 32 / NB;                        // pages a warp takes at once
    constexpr int IT = kPages / (kWarps * PW);         // times it does
    // query codes [hpk][NB] of 8 words positive, 8 negative and dq; blocks kBlock
    // words apart, so that lanes of different blocks read different banks; then the
    // pick's keys
    extern __shared__ __align__(16) uint32_t s_dyn[];
    __shared__ int s_last;
    uint32_t* s_q = s_dyn;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int e = blockIdx.z, kh = blockIdx.y;
    const int seq = e / a.T, t = e - seq * a.T;
    wait_for_earlier();
    let_next_start();
    const int np = page_count(a, seq, t, blockIdx.x == 0 && kh == 0 && tid == 0);
    const int p0 = blockIdx.x * kPages;
    int* out = a.pages + ((long long)e * a.g.Hkv + kh) * a.keep;
    if (blockIdx.x == 0)
        for (int i = min(a.keep, np) + tid; i < a.keep; i += kThreads) out[i] = -1;
    if (np <= a.keep) {                                // all pages: no scores
        if (blockIdx.x == 0)
            for (int i = tid; i < np; i += kThreads) out[i] = i;
        return;
    }
    if (p0 >= np) return;
    // page numbers and bounds of this lane's pages, on their way while the
    // query is coded
    const int* table = a.tables + (long long)seq * a.g.max_pages;
    const int b = lane % NB, pl = lane / NB;
    const int pe = min(np, p0 + kPages);
    int pg[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int p = p0 + (i * kWarps + warp) * PW + pl;
        pg[i] = p < pe ? table[p] : -2;
    }
    for (int i = warp; i < a.hpk * NB; i += kWarps) {  // a warp codes a block at a time
        const int h = kh * a.hpk + i / NB, bb = i - (i / NB) * NB;
        const long long at = ((long long)e * a.Hq + h) * D + 32 * bb + lane;
        const float x = a.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[at])
                               : reinterpret_cast<const float*>(a.q)[at];
        const float am = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(x))));
        const float inv = am > 0.f ? __fmul_rn(__frcp_rn(am), 127.f) : 0.f;
        const int c = (int)rintf(__fmul_rn(x, inv));
        int8_t* dst = reinterpret_cast<int8_t*>(s_q + (size_t)i * kBlock);
        dst[lane] = (int8_t)max(min(c, 127), 0);
        dst[32 + lane] = (int8_t)min(max(c, -127), 0);
        if (lane == 0) s_q[(size_t)i * kBlock + 16] = __float_as_uint(__fmul_rn(am, 1.0f / 127.0f));
    }
    __syncthreads();
    uint32_t* keys = a.keys + ((long long)e * a.g.Hkv + kh) * a.key_stride;
#pragma unroll 2
    for (int i = 0; i < IT; ++i) {
        const int p = p0 + (i * kWarps + warp) * PW + pl;
        const bool ok = pg[i] >= 0 && pg[i] < a.g.n_pages;
        uint32_t mn[8] = {}, mx[8] = {};
        float ds = 0.f;
        if (ok) {
            const long long at = ((long long)pg[i] * a.g.Hkv + kh) * NB + b;
            const uint4* src = reinterpret_cast<const uint4*>(a.codes + at * 64);
            const uint4 v0 = src[0], v1 = src[1], v2 = src[2], v3 = src[3];
            mn[0] = v0.x; mn[1] = v0.y; mn[2] = v0.z; mn[3] = v0.w; mn[4] = v1.x; mn[5] = v1.y; mn[6] = v1.z; mn[7] = v1.w;
            mx[0] = v2.x; mx[1] = v2.y; mx[2] = v2.z; mx[3] = v2.w; mx[4] = v3.x; mx[5] = v3.y; mx[6] = v3.z; mx[7] = v3.w;
            ds = a.scales[at];
        }
        float best = -__builtin_huge_valf();
        for (int q = 0; q < a.hpk; ++q) {
            const uint32_t* w = s_q + ((size_t)q * NB + b) * kBlock;
            const uint4 w0 = *reinterpret_cast<const uint4*>(w), w1 = *reinterpret_cast<const uint4*>(w + 4);
            const uint4 w2 = *reinterpret_cast<const uint4*>(w + 8), w3 = *reinterpret_cast<const uint4*>(w + 12);
            const uint32_t qp[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            const uint32_t qn[8] = {w2.x, w2.y, w2.z, w2.w, w3.x, w3.y, w3.z, w3.w};
            int d0 = 0, d1 = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                d0 = __dp4a((int)qp[k], (int)mx[k], d0);
                d1 = __dp4a((int)qn[k], (int)mn[k], d1);
            }
            const float part = __fmul_rn(__fmul_rn(__uint_as_float(w[16]), ds), (float)(d0 + d1));
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NB; ++k) s = __fadd_rn(s, __shfl_sync(0xffffffffu, part, pl * NB + k));
            best = fmaxf(best, s);
        }
        if (p < pe && b == 0) {
            if (!ok) atomicExch(a.g.err, kErrCounter);
            keys[p] = ok ? ordered(best) : 0u;
        }
    }
    // the last CTA of the (entry, KV head) picks
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const int n = (np + kPages - 1) / kPages;
        int* cnt = a.arrived + (long long)e * a.g.Hkv + kh;
        s_last = n == 1 || atomicAdd(cnt, 1) == n - 1;
        if (s_last && n > 1) *cnt = 0;
        __threadfence();
    }
    __syncthreads();
    if (s_last) pick(a, keys, s_dyn, np, out);
}

}  // namespace

template <int NB>
static cudaError_t launch_t(const SelectArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = kernel_attrs_once(select_kernel<NB>, done, false);
    if (e != cudaSuccess) return e;
    const size_t codes = (size_t)a.hpk * NB * kBlock * 4, keys = (size_t)std::min(a.key_stride, kKeep) * 4;
    const dim3 grid((unsigned)((a.g.max_pages + kPages - 1) / kPages), (unsigned)a.g.Hkv, (unsigned)(a.n_seq * a.T));
    return launch_dependent(select_kernel<NB>, grid, kThreads, std::max(codes, keys), s, a);
}

cudaError_t launch_select(const SelectArgs& a, cudaStream_t s) {
    switch (a.g.NB()) {
        case 2: return launch_t<2>(a, s);
        case 4: return launch_t<4>(a, s);
        default: return launch_t<8>(a, s);
    }
}

}  // namespace paged
}  // namespace kvq
