// Verification of drafted tokens (include/kvq.h, kvq_verify).
//
// Mathematics.  Draft d_t of a sequence stands while u_t q_t(d_t) < p_t(d_t); the
// products of two f32 numbers are exact in f64, so the test is one of real
// numbers; p and q are clean() first, as they are where they are summed.  At row a, the first whose draft falls or is none, the next token is
// drawn from weights w_i = max(P_i - Q_i, 0) (P_i where no draft stood), P and Q
// the probabilities in whole units of 2^-52: with S their sum it is the first i
// whose running sum passes floor(S u).  Sums of whole numbers do not depend on
// their order, so the row may be cut anywhere and the token stays the same, run
// by run and cut by cut; f32 sums over a row of 2^17 are off by more than its
// smaller probabilities.
//
// A cluster of blocks shares a row: each sums its part (every warp a stretch of
// it), the blocks tell each other their sums, and the one in whose part the
// running sum passes goes down into it: a warp's stretch is cut over all warps until
// 2048 elements are left, eight a thread at most, whose running sums end it.  One row
// of p and q is read of T; the parts read again come from L2.
//
// Measured: 64 sequences of 8 rows of 131072 tokens, f32, 17 us where the 67 MB take
// 10: 2.7 us until the row is known (two dependent loads), 8 of reading, then the
// slowest block of each cluster, its barrier and the last step, 1 each.  One
// sequence of 32000 tokens 5 us.  With sums by the exponent's shifts the integer pipe was the bound (21 us); loads
// of the next turn ahead of the sums cost registers and so blocks an SM (26 us).
#include "../../include/kvq.h"
#include "kvq_cluster.cuh"
#include "kvq_error.h"

#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 8;               // elements of a thread in the last step
using u64 = unsigned long long;

struct Args {
    const void* target;
    const void* draft;
    const int* tokens;
    const float* uniform;
    long long target_seq, target_row, draft_seq, draft_row;
    int T, vocab;
    int* accept;
    int* next;
    int* lens;
};

template <bool BF16>
__device__ __forceinline__ float element(const void* row, long long i) {
    if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
    else return reinterpret_cast<const float*>(row)[i];
}
template <bool BF16>
__device__ __forceinline__ const void* row_at(const void* base, long long i) {
    return reinterpret_cast<const uint8_t*>(base) + i * (BF16 ? 2 : 4);
}

// A probability in units of 2^-52, rounded down (0 where it is not above 0, NaN too, 1
// where it is above 1), as 22 + 15 + 15 bits in the low bits of three floats above
// 2^23: x 2^22 + 2^23 rounded down leaves the first, what that leaves out is exact,
// and so on.  That is eight operations of the multiply-add pipe a number, where shifts
// and masks by the exponent take ten of the integer pipe at half its rate; and sums of
// the floats' bits are sums of the parts, for the offsets of a p and a q cancel.
struct Parts {
    uint32_t h, m, l;
};
constexpr uint32_t kBase = 0x4b000000u;                  // of 2^23
__device__ __forceinline__ float clean(float x) {        // in [0, 1], of a NaN 0
    asm("add.sat.f32 %0, %1, 0f00000000;" : "=f"(x) : "f"(x));
    return x;
}
__device__ __forceinline__ Parts parts(float x) {        // (clean)
    const float base = 8388608.f;
    const float h = __fmaf_rz(x, 4194304.f, base);
    x = __fmaf_rn(x, 4194304.f, base - h);
    const float m = __fmaf_rz(x, 32768.f, base);
    x = __fmaf_rn(x, 32768.f, base - m);
    return {__float_as_uint(h), __float_as_uint(m), __float_as_uint(__fmaf_rz(x, 32768.f, base))};
}
__device__ __forceinline__ u64 units(float x) {
    const Parts p = parts(clean(x));
    return ((u64)(p.h - kBase) << 30) + ((p.m - kBase) << 15) + (p.l - kBase);
}

// Sums of up to 256 weights in three parts
struct Sum3 {
    uint32_t h = 0, m = 0, l = 0;
    // p less q, where that is above 0 (p > q: then P >= Q)
    __device__ __forceinline__ void add(float p, float q) {
        p = clean(p);
        q = clean(q);
        const Parts x = parts(p), y = parts(q);
        if (p > q) {
            h += x.h - y.h;
            m += x.m - y.m;
            l += x.l - y.l;
        }
    }
    __device__ __forceinline__ void add(float p) {
        const Parts x = parts(clean(p));
        h += x.h - kBase;
        m += x.m - kBase;
        l += x.l - kBase;
    }
    __device__ __forceinline__ u64 all() const { return ((u64)h << 30) + (u64)((long long)(int)m << 15) + (u64)(long long)(int)l; }
};

// What an element weighs: by p less q, or by p alone.  out: a lone draft's element, which weighs nothing
template <bool Q>
__device__ __forceinline__ u64 weight(float p, float q, bool out) {
    if constexpr (Q) {
        const long long w = (long long)(units(p) - units(q));
        return (u64)(w & ~(w >> 63));
    } else {
        return out ? 0ull : units(p);
    }
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The weights of [lo, hi) by one warp, a lane's share.  lo and hi are multiples of
// 32 (or the row's end); vec: both rows start on 16 bytes
template <bool BF16, bool Q>
__device__ __forceinline__ u64 sum_range(const void* p, const void* q, int lo, int hi, int tok, bool vec, int lane) {
    constexpr int V = BF16 ? 8 : 4, U = Q ? 4 : 8;       // elements of a load, loads of a row in flight
    u64 s = 0;
    int i = lo;
    auto step = [&](auto u) {
        constexpr int N = decltype(u)::value;
        uint4 a[N];
        [[maybe_unused]] uint4 b[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const long long at = i + (k * 32 + lane) * V;
            a[k] = __ldg(reinterpret_cast<const uint4*>(row_at<BF16>(p, at)));
            if constexpr (Q) b[k] = __ldg(reinterpret_cast<const uint4*>(row_at<BF16>(q, at)));
        }
        Sum3 t;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t x[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
            [[maybe_unused]] uint32_t y[4] = {};
            if constexpr (Q) y[0] = b[k].x, y[1] = b[k].y, y[2] = b[k].z, y[3] = b[k].w;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if constexpr (BF16) {
                    const float p0 = __uint_as_float(x[w] << 16), p1 = __uint_as_float(x[w] & 0xffff0000u);
                    if constexpr (Q) {
                        t.add(p0, __uint_as_float(y[w] << 16));
                        t.add(p1, __uint_as_float(y[w] & 0xffff0000u));
                    } else {
                        t.add(p0);
                        t.add(p1);
                    }
                } else {
                    if constexpr (Q) t.add(__uint_as_float(x[w]), __uint_as_float(y[w]));
                    else t.add(__uint_as_float(x[w]));
                }
            }
        }
        s += t.all();
        i += N * V * 32;
    };
    if (vec) {
        while (i + U * V * 32 <= hi) step(std::integral_constant<int, U>{});
        while (i + V * 32 <= hi) step(std::integral_constant<int, 1>{});
    }
    // element by element: rows that start anywhere, and what is left of a row
    constexpr int W = 8;
    for (; i < hi; i += W * 32) {
        float x[W], y[W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int at = i + k * 32 + lane;
            x[k] = at < hi ? element<BF16>(p, at) : 0.f;
            y[k] = Q && at < hi ? element<BF16>(q, at) : 0.f;
        }
        Sum3 t;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if constexpr (Q) t.add(x[k], y[k]);
            else t.add(x[k]);
        }
        s += t.all();
    }
    // (a sum of whole numbers: what a lone draft's element brought is taken off again)
    if (!Q && lane == 0 && tok >= lo && tok < hi) s -= units(element<BF16>(p, tok));
    return s;
}

// Sequence blockIdx.x / C by a cluster of C blocks
template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ Args a) {
    __shared__ int s_row, s_held, s_tok;
    __shared__ u64 s_sum[kWarps];
    __shared__ u64 s_all[2][cluster::kMaxCluster];       // the blocks' sums, written by themselves
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = cluster::size(), rank = cluster::rank();
    const long long b = blockIdx.x / C;
    cluster::arrive();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- the first draft that does not stand
    if (warp == 0) {
        int row = a.T - 1, tok = -1;
        for (int t0 = 0; t0 < a.T - 1; t0 += 32) {
            const int t = t0 + lane;
            int d = -1;
            bool ok = false;
            if (t < a.T - 1) {
                d = a.tokens[b * (a.T - 1) + t];
                if (d >= 0 && d < a.vocab) {
                    const float p = clean(element<BF16>(a.target, b * a.target_seq + t * a.target_row + d));
                    const float q = a.draft ? clean(element<BF16>(a.draft, b * a.draft_seq + t * a.draft_row + d)) : 1.f;
                    ok = (double)a.uniform[b * a.T + t] * (double)q < (double)p;
                } else {
                    d = -1;
                }
            }
            const unsigned no = __ballot_sync(0xffffffffu, t < a.T - 1 && !ok);
            if (no) {
                const int l = __ffs(no) - 1;
                row = t0 + l;
                tok = __shfl_sync(0xffffffffu, d, l);
                break;
            }
        }
        if (lane == 0) {
            s_row = row;
            s_held = tok >= 0;                           // a draft stood here: its share is taken off
            s_tok = tok;
            if (rank == 0) {
                a.accept[b] = row + 1;
                a.next[b] = -1;                          // (the block that finds the token writes it behind the cluster's barrier)
                if (a.lens) a.lens[b] -= a.T - 1 - row;
            }
        }
    }
    __syncthreads();
    const int row = s_row;
    bool with_q = s_held && a.draft;
    int tok = s_held && !a.draft ? s_tok : -1;
    const void* p = row_at<BF16>(a.target, b * a.target_seq + row * a.target_row);
    const void* q = with_q ? row_at<BF16>(a.draft, b * a.draft_seq + row * a.draft_row) : p;
    const bool vec = (((uintptr_t)p | (uintptr_t)q) & 15) == 0;
    // ---- sums of this block's part; where nothing is left of p over q, of p itself
    auto part = [](int n, int parts) { return ((n + parts - 1) / parts + 31) & ~31; };
    int lo = min(a.vocab, rank * part(a.vocab, C)), hi = min(a.vocab, lo + part(a.vocab, C));
    int per = part(hi - lo, kWarps);
    auto sums = [&](int from, int to) {
        const int x = min(to, from + warp * per), y = min(to, x + per);
        const u64 s = warp_sum(with_q ? sum_range<BF16, true>(p, q, x, y, -1, vec, lane) : sum_range<BF16, false>(p, q, x, y, tok, vec, lane));
        if (lane == 0) s_sum[warp] = s;
        __syncthreads();
    };
    u64 S = 0, first = 0, mine = 0;
    for (int mode = 0; mode < 2; ++mode) {
        sums(lo, hi);
        if (mode == 0) cluster::started();
        if (tid < C) {
            u64 t = 0;
            for (int w = 0; w < kWarps; ++w) t += s_sum[w];
            cluster::store(cluster::map(&s_all[mode][rank], tid), t);
        }
        cluster::sync();
        for (int r = 0; r < C; ++r) {
            if (r == rank) first = S;
            S += s_all[mode][r];
        }
        mine = s_all[mode][rank];
        if (S != 0) break;                               // (the same in all blocks of the cluster)
        with_q = false;
        tok = -1;
    }
    if (S == 0) return;
    const float u = a.uniform[b * a.T + a.T - 1];
    const uint32_t U = u > 0.f ? (uint32_t)fminf(u * 2147483648.f, 2147483520.f) : 0u;   // (the f32 below 2^31)
    u64 x = __umul64hi(S, (u64)U << 33);                 // floor(S U 2^-31)
    if (x < first || x - first >= mine) return;
    x -= first;
    // ---- down into the stretch where the running sum passes x
    for (;;) {
        int w = 0;
        while (w < kWarps - 1 && x >= s_sum[w]) x -= s_sum[w++];
        lo = min(hi, lo + w * per);
        hi = min(hi, lo + per);
        __syncthreads();                                 // (before the sums are written again)
        if (hi - lo <= kEach * kThreads) break;
        per = part(hi - lo, kWarps);
        sums(lo, hi);
    }
    const int each = (hi - lo + kThreads - 1) / kThreads, i0 = lo + tid * each;
    u64 v[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = i0 + k;
        v[k] = 0;
        if (k < each && i < hi) v[k] = with_q ? weight<true>(element<BF16>(p, i), element<BF16>(q, i), false) : weight<false>(element<BF16>(p, i), 0.f, i == tok);
        sum += v[k];
    }
    u64 run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    if (lane == 31) s_sum[warp] = run;
    __syncthreads();
    u64 at = run - sum;                                  // before this thread's elements
    for (int w = 0; w < warp; ++w) at += s_sum[w];
    if (x < at || x - at >= sum) return;                 // (one thread goes on)
    int found = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        at += v[k];
        found += at <= x;
    }
    a.next[b] = min(i0 + found, a.vocab - 1);
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_verify(const kvq_verify_args* v, void* stream) {
    if (!v) return fail(KVQ_EINVAL, "args is NULL");
    if (v->dtype != KVQ_F32 && v->dtype != KVQ_BF16) return fail(KVQ_EINVAL, "dtype must be f32 or bf16");
    if (v->n_seq < 1 || v->n_seq > 65536) return fail(KVQ_EINVAL, "n_seq=%d outside [1, 65536]", v->n_seq);
    if (v->T < 1 || v->T > 512) return fail(KVQ_EINVAL, "T=%d outside [1, 512]", v->T);
    if (v->vocab < 1 || v->vocab > (1 << 24)) return fail(KVQ_EINVAL, "vocab=%d outside [1, 2^24]", v->vocab);
    if (!v->target || !v->uniform || !v->accept || !v->next) return fail(KVQ_EINVAL, "target, uniform, accept or next is NULL");
    if (v->T > 1 && !v->tokens) return fail(KVQ_EINVAL, "tokens is NULL");
    const size_t size = v->dtype == KVQ_BF16 ? 2 : 4;
    if ((size_t)v->target % size || (size_t)v->draft % size || ((size_t)v->tokens | (size_t)v->uniform | (size_t)v->accept | (size_t)v->next | (size_t)v->lens) % 4)
        return fail(KVQ_EINVAL, "a pointer is not aligned to its elements");
    if (v->target_seq < 0 || v->target_row < 0 || v->draft_seq < 0 || v->draft_row < 0)
        return fail(KVQ_EINVAL, "strides must be >= 0");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    static std::atomic<int> known[64];                   // SMs of each device, asked for once
    int sms = known[dev & 63].load(std::memory_order_relaxed);
    if (sms == 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        known[dev & 63].store(sms, std::memory_order_relaxed);
    }
    Args a{v->target, v->draft, v->tokens, v->uniform, v->target_seq, v->target_row, v->draft_seq, v->draft_row,
           v->T, v->vocab, v->accept, v->next, v->lens};
    // blocks of a row: more while SMs are idle and a part keeps some 2000 elements
    int C = 1;
    while (C < cluster::kMaxCluster && (long long)v->n_seq * C < 4LL * sms && v->vocab > 2048 * C) C *= 2;
    const dim3 grid((unsigned)(v->n_seq * C));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = v->dtype == KVQ_BF16 ? cluster::launch(verify_kernel<true>, grid, C, kThreads, 0, s, a)
                             : cluster::launch(verify_kernel<false>, grid, C, kThreads, 0, s, a);
    return e == cudaSuccess ? KVQ_OK : cuda_fail(e, "verify kernel");
}
