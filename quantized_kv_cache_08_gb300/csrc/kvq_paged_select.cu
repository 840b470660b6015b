// Choosing the pages that a query reads, by the key bounds of the pages.
//
// A page's score is an upper bound of the query's product with every key in it:
// sum over elements of max(c min, c max) for the query code c, which is c max
// where c > 0 and c min elsewhere, so two integer dot products of the query's
// positive and negative parts give it exactly; the two scales and the sum over
// blocks are single f32 operations in a fixed order.  Scores are therefore the
// same numbers on every run, and ties (common between codes) go to the lowest
// index.  Two kernels: scores, then the largest `keep` by a radix search for
// the threshold, eight bits a pass, and a compaction in index order.
#include "kvq_paged.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSelThreads = 512;
constexpr uint32_t kForced = 0xffffffffu;

// number of pages with a row that query row t sees, -1 for a bad length
__device__ __forceinline__ int page_count(const SelectArgs& a, int seq, int t, bool report) {
    const int len = a.lens[seq];
    if (len < 0 || len > (long long)a.g.max_pages << a.g.page_shift) {
        if (report) atomicExch(a.g.err, kErrCounter);
        return 0;
    }
    const int hi = len - a.T + t + 1;
    return hi > 0 ? (hi + a.g.page_rows - 1) >> a.g.page_shift : 0;
}

// f32 -> an unsigned integer of the same order (-0 counts as 0), below kForced
__device__ __forceinline__ uint32_t ordered(float s) {
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Scores of pages [PB blockIdx.x, + PB) for KV head blockIdx.y and entry
// blockIdx.z: NB lanes a page, one 32-element block each.
template <int NB>
__global__ void __launch_bounds__(kThreads) score_kernel(const SelectArgs a, int PB) {
    constexpr int D = NB * 32;
    constexpr int PW = 32 / NB;                        // pages a warp takes at once
    extern __shared__ __align__(16) uint32_t s_q[];    // [hpk][NB][8 words positive, 8 words negative], then dq [hpk][NB]
    float* s_dq = reinterpret_cast<float*>(s_q + (size_t)a.hpk * NB * 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int e = blockIdx.z, kh = blockIdx.y;
    const int seq = e / a.T, t = e - seq * a.T;
    const int np = page_count(a, seq, t, blockIdx.x == 0 && kh == 0 && tid == 0);
    const int p0 = blockIdx.x * PB;
    if (p0 >= np) return;
    // query codes: a warp takes a block at a time
    for (int i = warp; i < a.hpk * NB; i += kWarps) {
        const int h = kh * a.hpk + i / NB, b = i - (i / NB) * NB;
        const long long at = ((long long)e * a.Hq + h) * D + 32 * b + lane;
        const float x = a.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[at])
                               : reinterpret_cast<const float*>(a.q)[at];
        float am = fabsf(x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        const float inv = am > 0.f ? __fmul_rn(__frcp_rn(am), 127.f) : 0.f;
        const int c = (int)rintf(__fmul_rn(x, inv));
        int8_t* dst = reinterpret_cast<int8_t*>(s_q + (size_t)i * 16);
        dst[lane] = (int8_t)max(min(c, 127), 0);
        dst[32 + lane] = (int8_t)min(max(c, -127), 0);
        if (lane == 0) s_dq[i] = __fmul_rn(am, 1.0f / 127.0f);
    }
    __syncthreads();
    const int* table = a.tables + (long long)seq * a.g.max_pages;
    uint32_t* keys = a.keys + ((long long)e * a.g.Hkv + kh) * a.g.max_pages;
    const int b = lane % NB, pl = lane / NB;
    const int pe = min(np, p0 + PB);
    for (int pb = p0 + warp * PW; pb < pe; pb += kWarps * PW) {
        const int p = pb + pl;
        bool ok = p < pe;
        int pg = ok ? table[p] : 0;
        if (ok && (pg < 0 || pg >= a.g.n_pages)) {
            atomicExch(a.g.err, kErrCounter);
            ok = false;
        }
        uint32_t mn[8] = {}, mx[8] = {};
        float ds = 0.f;
        if (ok) {
            const long long at = ((long long)pg * a.g.Hkv + kh) * NB + b;
            const uint4* src = reinterpret_cast<const uint4*>(a.codes + at * 64);
            const uint4 v0 = src[0], v1 = src[1], v2 = src[2], v3 = src[3];
            mn[0] = v0.x; mn[1] = v0.y; mn[2] = v0.z; mn[3] = v0.w; mn[4] = v1.x; mn[5] = v1.y; mn[6] = v1.z; mn[7] = v1.w;
            mx[0] = v2.x; mx[1] = v2.y; mx[2] = v2.z; mx[3] = v2.w; mx[4] = v3.x; mx[5] = v3.y; mx[6] = v3.z; mx[7] = v3.w;
            ds = a.scales[at];
        }
        float best = -__builtin_huge_valf();
        for (int q = 0; q < a.hpk; ++q) {
            const uint4* w = reinterpret_cast<const uint4*>(s_q + ((size_t)q * NB + b) * 16);
            const uint4 w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
            const uint32_t qp[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            const uint32_t qn[8] = {w2.x, w2.y, w2.z, w2.w, w3.x, w3.y, w3.z, w3.w};
            int dot = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dot = __dp4a((int)qp[i], (int)mx[i], dot);
                dot = __dp4a((int)qn[i], (int)mn[i], dot);
            }
            const float part = __fmul_rn(__fmul_rn(s_dq[q * NB + b], ds), (float)dot);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) s = __fadd_rn(s, __shfl_sync(0xffffffffu, part, pl * NB + i));
            best = fmaxf(best, s);
        }
        if (p < pe && b == 0) {
            uint32_t key = ok ? ordered(best) : 0u;
            if (p < a.n_first || p >= np - a.n_last) key = kForced;
            keys[p] = key;
        }
    }
}

// The `keep` largest keys of one (entry, KV head), ties to the lowest index.
__global__ void __launch_bounds__(kSelThreads) pick_kernel(const SelectArgs a) {
    __shared__ int s_hist[256];
    __shared__ int s_wsum[kSelThreads / 32], s_weq[kSelThreads / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int e = blockIdx.y, kh = blockIdx.x;
    const int seq = e / a.T, t = e - seq * a.T;
    const int np = page_count(a, seq, t, false);
    const uint32_t* keys = a.keys + ((long long)e * a.g.Hkv + kh) * a.g.max_pages;
    int* out = a.pages + ((long long)e * a.g.Hkv + kh) * a.keep;
    const int keep = min(a.keep, np);
    for (int i = keep + tid; i < a.keep; i += kSelThreads) out[i] = -1;
    if (keep == np) {
        for (int i = tid; i < keep; i += kSelThreads) out[i] = i;
        return;
    }
    uint32_t prefix = 0;
    int need = keep;                                    // keys still to find among those that share the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int i = tid; i < np; i += kSelThreads) {
            const uint32_t k = keys[i];
            if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1);
        }
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
                while (before + c[i] < need) before += c[i++];
                s_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
                s_need = need - before;
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    }
    // keys above the threshold and the first `need` that equal it, in order
    int done = 0, eq_done = 0;
    for (int base = 0; base < np; base += kSelThreads) {
        const int i = base + tid;
        const uint32_t k = i < np ? keys[i] : 0u;
        const bool gt = i < np && k > prefix, eq = i < np && k == prefix;
        const unsigned me = __ballot_sync(0xffffffffu, eq), mg = __ballot_sync(0xffffffffu, gt);
        const unsigned below = (1u << lane) - 1u;
        if (lane == 0) {
            s_weq[warp] = __popc(me);
            s_wsum[warp] = __popc(mg);
        }
        __syncthreads();
        int eb = eq_done, gb = done, et = 0, gt_all = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) {
            if (w < warp) {
                eb += s_weq[w];
                gb += s_wsum[w];
            }
            et += s_weq[w];
            gt_all += s_wsum[w];
        }
        const int erank = eb + __popc(me & below);       // equal keys before this one
        // taken before this one: greater keys, and equal ones up to `need`
        const int at = gb + __popc(mg & below) + min(erank, need);
        if (gt || (eq && erank < need)) out[at] = i;
        done += gt_all;
        eq_done += et;
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, cudaStream_t s) {
    const int E = a.n_seq * a.T, nb = a.g.NB();
    const int PB = 64;
    const dim3 grid((unsigned)((a.g.max_pages + PB - 1) / PB), (unsigned)a.g.Hkv, (unsigned)E);
    const size_t smem = (size_t)a.hpk * nb * (16 * 4 + 4);
    if (smem > 48 * 1024) {                              // 128 queries a KV head at head_dim 256: 68 KB
        static std::atomic<unsigned long long> d2{0}, d4{0}, d8{0};
        cudaError_t e = nb == 2 ? kernel_attrs_once(score_kernel<2>, d2, false)
                      : nb == 4 ? kernel_attrs_once(score_kernel<4>, d4, false)
                                : kernel_attrs_once(score_kernel<8>, d8, false);
        if (e != cudaSuccess) return e;
    }
    if (nb == 2) score_kernel<2><<<grid, kThreads, smem, s>>>(a, PB);
    else if (nb == 4) score_kernel<4><<<grid, kThreads, smem, s>>>(a, PB);
    else score_kernel<8><<<grid, kThreads, smem, s>>>(a, PB);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    pick_kernel<<<dim3((unsigned)a.g.Hkv, (unsigned)E), kSelThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace paged
}  // namespace kvq
