// Host side of the paged-cache calls: validation, workspace layout, launches.
// See include/kvq.h for the contract of every entry point.
#include "../../include/kvq.h"
#include "kvq_error.h"
#include "kvq_paged.cuh"

#include <algorithm>
#include <cmath>
#include <new>

using namespace kvq;
using namespace kvq::paged;

struct kvq_paged {
    kvq_paged_config cfg;
    Geom g;
    int num_sms;
    uint8_t* ws;
    size_t off_plan, off_plan2, off_arrived, off_ml, off_o, off_ml2, off_o2, off_keys, key_rows, keys2;
    int8_t* codes;
    float* scales;
    Freqs freqs;
};

namespace {

constexpr int kMaxGrid = 256;          // most CTAs of a split kernel
constexpr int kMaxRanges = 4 * kMaxGrid;
// Keys from which groups of four warps work on ranges of their own.  16: 47 us for
// 32 f32 queries over 16k rows of 4 KV heads of 256 (16 keys), 32 and 64: 40; a
// window over 7 sequences of 8 KV heads of 64 (56 keys) 17 us, at 64: 22.  At head_dim
// 256 a CTA has two groups only, which hide less of each other: 4 sequences of 32768
// rows there (32 keys) 127 us, at 64: 118.
constexpr int many_keys(int NB) { return NB == 8 ? 64 : 32; }
// what a change of key costs a group of warps, in cells.  8: 196 us for a batch
// of 64 (1024 to 16k rows, 8 KV heads of 128), 24: 189, 48: 193; a window of 4096
// rows over 7 sequences 21.3, 17.2, 17.8
constexpr int kSetup = 24;
constexpr int kMaxT = 64;
constexpr int kMaxRows = 1 << 24;      // rows of a sequence at most

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned16(const void* p) { return ((size_t)p & 15) == 0; }

struct Layout {
    size_t cell, page, pool, bounds, plan, plan2, arrived, ml, o, ml2, o2, keys, total, key_rows, keys2;
};

kvq_status layout(const kvq_paged_config* c, Layout* l) {
    if (!c) return fail(KVQ_EINVAL, "config is NULL");
    const bool q8q5 = c->k_fmt == KVQ_Q8_0 && c->v_fmt == KVQ_Q5_1;
    const bool f8 = c->k_fmt == KVQ_FP8_E4M3 && c->v_fmt == KVQ_FP8_E4M3;
    if (!q8q5 && !f8) return fail(KVQ_EUNSUPPORTED, "formats must be K=q8_0, V=q5_1 or K=V=fp8_e4m3");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(KVQ_EUNSUPPORTED, "a paged cache takes head_dim 64, 128 or 256");
    const int R = c->page_rows;
    if (R != 16 && R != 32 && R != 64 && R != 128 && R != 256)
        return fail(KVQ_EINVAL, "page_rows must be 16, 32, 64, 128 or 256");
    if (c->n_pages < 1) return fail(KVQ_EINVAL, "n_pages must be >= 1");
    if (c->n_kv_heads < 1 || c->n_kv_heads > 128) return fail(KVQ_EINVAL, "n_kv_heads must be in [1, 128]");
    if (c->max_q_heads < c->n_kv_heads || c->max_q_heads % c->n_kv_heads || c->max_q_heads / c->n_kv_heads > 128)
        return fail(KVQ_EINVAL, "max_q_heads must be a multiple of n_kv_heads, at most 128 times it");
    if (c->max_seqs < 1 || c->max_seqs > kMaxSeqs) return fail(KVQ_EINVAL, "max_seqs must be in [1, %d]", kMaxSeqs);
    if (c->max_pages < 1 || (long long)c->max_pages * R > kMaxRows)
        return fail(KVQ_EINVAL, "max_pages must be >= 1 and max_pages * page_rows at most 2^24");
    if (c->max_t < 1 || c->max_t > kMaxT) return fail(KVQ_EINVAL, "max_t must be in [1, %d]", kMaxT);
    if (c->rope_dim < 0 || c->rope_dim > c->head_dim || c->rope_dim % 16)
        return fail(KVQ_EINVAL, "rope_dim must be 0 or a multiple of 16 up to head_dim");
    const size_t NB = c->head_dim / 32, D = c->head_dim;
    l->cell = NB * (f8 ? 1024 : 928);
    l->page = l->cell * (R / kCellRows) * c->n_kv_heads;
    l->pool = l->page * c->n_pages;
    l->bounds = c->bounds ? round_up((size_t)c->n_pages * c->n_kv_heads * NB * 68, 16) : 0;
    // record rows of a decode: 16 (or 8) for each range, each key of
    // a sequence in whole slices, and the groups' queries, which are their
    // members', in whole slices too
    const size_t Qh = (size_t)(c->max_q_heads / c->n_kv_heads) * c->max_t;
    l->key_rows = (size_t)c->n_kv_heads * c->max_seqs * (round_up(Qh, 16) + Qh + 16);
    const size_t recs = (size_t)kMaxRanges * 16 + l->key_rows;
    l->plan = 256;                                       // the error word comes first
    l->plan2 = round_up(l->plan + (kMaxEntries + 1) * sizeof(PlanEntry), 256);
    l->arrived = round_up(l->plan2 + (kMaxSeqs + 1) * sizeof(PlanEntry), 256);
    l->ml = round_up(l->arrived + l->key_rows * sizeof(int), 256);
    l->o = round_up(l->ml + recs * 8, 256);
    // records of the prefix tile kernel: tile_rows queries for each CTA and each
    // key; groups that it takes have more than 8 queries each
    const size_t tr = prefix_rows_of((int)NB);
    const size_t total_q = (size_t)c->max_seqs * Qh;
    l->keys2 = (size_t)c->n_kv_heads * (total_q / tr + std::min<size_t>(c->max_seqs, total_q / 9) + 1);
    const size_t recs2 = total_q > 8 ? (kMaxGrid + l->keys2) * tr : 0;
    l->ml2 = round_up(l->o + recs * D * 4, 256);
    l->o2 = round_up(l->ml2 + recs2 * 16, 256);
    l->keys = round_up(l->o2 + recs2 * D * 2, 256);
    l->total = l->keys;
    if (c->bounds)
        l->total += round_up((size_t)std::min(kMaxEntries, c->max_seqs * c->max_t) * c->n_kv_heads * round_up(c->max_pages, 4) * 4, 256);
    return KVQ_OK;
}

kvq_status check_rows(const kvq_paged* c, const int* tables, const int* lens, int n_seq, int T, const int* starts,
                      int rows, Rows* r) {
    if (!tables || !lens) return fail(KVQ_EINVAL, "tables or lens is NULL");
    if (n_seq < 1 || n_seq > c->cfg.max_seqs) return fail(KVQ_EINVAL, "n_seq=%d outside [1, max_seqs=%d]", n_seq, c->cfg.max_seqs);
    if (starts) {
        if (rows < 0) return fail(KVQ_EINVAL, "rows must be >= 0");
    } else {
        if (T < 1 || (long long)n_seq * T > 0x7fffffffLL) return fail(KVQ_EINVAL, "T=%d must be >= 1", T);
        if (rows != n_seq * T) return fail(KVQ_EINVAL, "rows=%d is not n_seq * T", rows);
    }
    if ((long long)rows * c->cfg.max_q_heads > (1LL << 31)) return fail(KVQ_ERANGE, "rows=%d too many for one call", rows);
    r->tables = tables;
    r->lens = lens;
    r->starts = starts;
    r->n_seq = n_seq;
    r->T = T;
    r->rows = rows;
    return KVQ_OK;
}

kvq_status check_stride(const char* what, const void* p, long long stride, long long dense) {
    if (!aligned16(p)) return fail(KVQ_EINVAL, "%s must be 16-byte aligned", what);
    if (stride < dense || stride % 8) return fail(KVQ_EINVAL, "%s_stride must be a multiple of 8 and at least %lld", what, dense);
    return KVQ_OK;
}

kvq_status bounds_of(kvq_paged* c, const Rows& r, cudaStream_t s) {
    BoundsArgs b{c->g, r, c->codes, c->scales};
    cudaError_t e = launch_bounds(b, s);
    return e == cudaSuccess ? KVQ_OK : cuda_fail(e, "page bounds kernel");
}

kvq_status check_query(const kvq_paged* c, const kvq_paged_query* a) {
    if (!c) return fail(KVQ_EINVAL, "cache is NULL");
    if (!a) return fail(KVQ_EINVAL, "query is NULL");
    if (!a->q || !a->tables || !a->lens) return fail(KVQ_EINVAL, "q, tables or lens is NULL");
    if (a->dtype != KVQ_F32 && a->dtype != KVQ_BF16) return fail(KVQ_EINVAL, "dtype must be f32 or bf16");
    if (a->n_seq < 1 || a->n_seq > c->cfg.max_seqs)
        return fail(KVQ_EINVAL, "n_seq=%d outside [1, max_seqs=%d]", a->n_seq, c->cfg.max_seqs);
    if (a->T < 1 || a->T > c->cfg.max_t) return fail(KVQ_EINVAL, "T=%d outside [1, max_t=%d]", a->T, c->cfg.max_t);
    const int Hkv = c->cfg.n_kv_heads;
    if (a->n_q_heads < Hkv || a->n_q_heads % Hkv || a->n_q_heads > c->cfg.max_q_heads)
        return fail(KVQ_EINVAL, "n_q_heads must be a multiple of n_kv_heads and <= max_q_heads");
    if (!aligned16(a->q)) return fail(KVQ_EINVAL, "q must be 16-byte aligned");
    return KVQ_OK;
}

kvq_status decode(kvq_paged* c, const kvq_paged_query* q, const int* group_start, const int* prefix_len, int n_groups,
                  const int* lists, int keep, void* stream) {
    kvq_status st = check_query(c, q);
    if (st != KVQ_OK) return st;
    if (!q->out || !aligned16(q->out)) return fail(KVQ_EINVAL, "out is NULL or not 16-byte aligned");
    // (both go through products and quotients in f32)
    if (!(q->softcap == 0.f || (q->softcap >= 1e-30f && q->softcap <= 1e30f)))
        return fail(KVQ_EINVAL, "softcap must be 0 or within 1e-30 .. 1e30");
    if (!(q->scale <= 0.f || (q->scale >= 1e-30f && q->scale <= 1e30f)))
        return fail(KVQ_EINVAL, "scale must be <= 0 (1 / sqrt(head_dim)) or within 1e-30 .. 1e30");
    if (q->window < 0) return fail(KVQ_EINVAL, "window must be >= 0");
    SplitArgs a = {};
    a.g = c->g;
    a.q = q->q;
    a.out = q->out;
    a.bf16 = q->dtype == KVQ_BF16;
    a.n_seq = q->n_seq;
    a.T = q->T;
    a.Hq = q->n_q_heads;
    a.hpk = q->n_q_heads / c->cfg.n_kv_heads;
    a.tables = q->tables;
    a.lens = q->lens;
    a.sinks = q->sinks;
    const float log2e = 1.4426950408889634f;
    a.qscale = (q->scale > 0.f ? q->scale : 1.0f / sqrtf((float)c->cfg.head_dim)) * log2e;
    a.softcap_a = q->softcap > 0.f ? 1.0f / (q->softcap * log2e) : 0.f;
    a.softcap_b = q->softcap > 0.f ? q->softcap * log2e : 0.f;
    // (a window of the longest sequence is none; positions less a larger one could pass 32 bits)
    a.window = std::min(q->window, kMaxRows);
    a.group_start = group_start;
    a.prefix_len = prefix_len;
    a.n_groups = n_groups;
    a.lists = lists;
    a.keep = keep;
    a.E = lists ? q->n_seq * q->T : q->n_seq + n_groups;
    a.G = std::min(c->num_sms, kMaxGrid);
    // queries of a key at most: the tile kernel takes the bf16 groups that have
    // more than a slice
    const int own = lists ? a.hpk : a.hpk * q->T;
    a.tile = split_tile(a.g.NB(), a.bf16, own);
    a.tiles = n_groups > 0 && a.bf16 && q->n_seq * own > a.tile;
    const int most = n_groups > 0 ? (a.tiles ? a.tile : q->n_seq * own) : own;
    // many keys: four warps a group, for a fragment's end and start are hidden
    // behind the other groups; few keys: the whole CTA, for a quarter of the
    // records to join
    const int warps = split_warps(a.g.NB(), a.tile);
    const long long keys = (long long)a.E * c->cfg.n_kv_heads * ((most + a.tile - 1) / a.tile);
    a.gw = keys >= many_keys(a.g.NB()) ? 4 : warps;
    a.groups = warps / a.gw;
    a.setup = kSetup;
    a.rec_rows = std::min(a.tile, most);
    a.max_keys = (long long)(c->key_rows / a.rec_rows);
    a.plan = reinterpret_cast<PlanEntry*>(c->ws + c->off_plan);
    a.arrived = reinterpret_cast<int*>(c->ws + c->off_arrived);
    a.fuse = n_groups == 0;
    a.part_ml = reinterpret_cast<float*>(c->ws + c->off_ml);
    a.part_o = reinterpret_cast<float*>(c->ws + c->off_o);
    a.tile_rows = prefix_rows_of(a.g.NB());
    a.max_keys2 = (long long)c->keys2;
    a.plan2 = reinterpret_cast<PlanEntry*>(c->ws + c->off_plan2);
    a.part2_ml = reinterpret_cast<float*>(c->ws + c->off_ml2);
    a.part2_o = reinterpret_cast<uint16_t*>(c->ws + c->off_o2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (a.tiles) {
        e = launch_prefix(a, s);
        if (e != cudaSuccess) return cuda_fail(e, "paged decode prefix kernel");
    }
    e = launch_split(a, s);
    if (e != cudaSuccess) return cuda_fail(e, "paged decode split kernel");
    if (!a.fuse) e = launch_merge(a, s);
    if (e != cudaSuccess) return cuda_fail(e, "paged decode merge kernel");
    return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_paged_required_bytes(const kvq_paged_config* cfg, kvq_paged_sizes* out) {
    Layout l;
    kvq_status st = layout(cfg, &l);
    if (st != KVQ_OK) return st;
    if (!out) return fail(KVQ_EINVAL, "out is NULL");
    out->pool = l.pool;
    out->bounds = l.bounds;
    out->workspace = l.total;
    out->page_bytes = l.page;
    out->cell_bytes = l.cell;
    return KVQ_OK;
}

kvq_status kvq_paged_alloc(const kvq_paged_config* cfg, void* pool, void* bounds, void* workspace,
                           const double* rope_freq, void* stream, kvq_paged** out) {
    Layout l;
    kvq_status st = layout(cfg, &l);
    if (st != KVQ_OK) return st;
    if (!out) return fail(KVQ_EINVAL, "out is NULL");
    *out = nullptr;
    if (!pool || !workspace || (cfg->bounds && !bounds)) return fail(KVQ_EINVAL, "a device buffer is NULL");
    if (!aligned16(pool) || !aligned16(bounds) || !aligned16(workspace))
        return fail(KVQ_EINVAL, "device buffers must be 16-byte aligned");
    if (cfg->rope_dim && !rope_freq && !(cfg->rope_base > 0.0 && std::isfinite(cfg->rope_base)))
        return fail(KVQ_EINVAL, "rope_base must be positive and finite");
    const double turn = 6.283185307179586476925;
    Freqs f = {};
    for (int i = 0; i < cfg->rope_dim / 2; ++i) {
        const double w = rope_freq ? rope_freq[i] : std::pow(cfg->rope_base, -2.0 * i / cfg->rope_dim);
        if (!(std::fabs(w) <= 64.0)) return fail(KVQ_EINVAL, "rope frequency %d is not within 64 radians a position", i);
        // whole turns a position are none: what is left is half a turn at most, of which
        // the two floats keep 2^-50 and the kernel's sums 2^-24 at any position
        const double turns = w / turn - std::nearbyint(w / turn);
        f.f[i].x = (float)turns;
        f.f[i].y = (float)(turns - (double)f.f[i].x);
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    // the error word, and the counters that every decode leaves at zero
    e = cudaMemsetAsync(workspace, 0, l.ml, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(workspace)");
    kvq_paged* c = new (std::nothrow) kvq_paged();
    if (!c) return fail(KVQ_ERANGE, "out of host memory");
    c->cfg = *cfg;
    c->g.pool = static_cast<uint8_t*>(pool);
    c->g.err = static_cast<int*>(workspace);
    c->g.n_pages = cfg->n_pages;
    c->g.page_rows = cfg->page_rows;
    c->g.page_shift = 0;
    while ((1 << c->g.page_shift) < cfg->page_rows) ++c->g.page_shift;
    c->g.max_pages = cfg->max_pages;
    c->g.Hkv = cfg->n_kv_heads;
    c->g.D = cfg->head_dim;
    c->g.fp8 = cfg->k_fmt == KVQ_FP8_E4M3;
    c->g.cell_bytes = (int)l.cell;
    c->g.page_bytes = (long long)l.page;
    c->num_sms = sms;
    c->ws = static_cast<uint8_t*>(workspace);
    c->off_plan = l.plan;
    c->off_plan2 = l.plan2;
    c->off_ml2 = l.ml2;
    c->off_o2 = l.o2;
    c->keys2 = l.keys2;
    c->off_arrived = l.arrived;
    c->off_ml = l.ml;
    c->off_o = l.o;
    c->off_keys = l.keys;
    c->key_rows = l.key_rows;
    c->codes = static_cast<int8_t*>(bounds);
    const size_t nb = (size_t)cfg->n_pages * cfg->n_kv_heads * (cfg->head_dim / 32);
    c->scales = bounds ? reinterpret_cast<float*>(static_cast<uint8_t*>(bounds) + nb * 64) : nullptr;
    c->freqs = f;
    *out = c;
    return KVQ_OK;
}

void kvq_paged_free(kvq_paged* cache) { delete cache; }

kvq_status kvq_paged_append(kvq_paged* c, const void* k, long long k_stride, const void* v, long long v_stride,
                            const void* q, long long q_stride, void* q_out, int n_q_heads, kvq_dtype dtype,
                            const int* tables, const int* lens, int n_seq, int T, const int* starts, int rows,
                            void* stream) {
    if (!c) return fail(KVQ_EINVAL, "cache is NULL");
    if (dtype != KVQ_F32 && dtype != KVQ_BF16) return fail(KVQ_EINVAL, "dtype must be f32 or bf16");
    AppendArgs a = {};
    kvq_status st = check_rows(c, tables, lens, n_seq, T, starts, rows, &a.r);
    if (st != KVQ_OK || rows == 0) return st;
    if (!k || !v) return fail(KVQ_EINVAL, "k or v is NULL");
    const long long kvd = (long long)c->cfg.n_kv_heads * c->cfg.head_dim;
    if ((st = check_stride("k", k, k_stride, kvd)) != KVQ_OK) return st;
    if ((st = check_stride("v", v, v_stride, kvd)) != KVQ_OK) return st;
    if (q) {
        if (!q_out || !aligned16(q_out)) return fail(KVQ_EINVAL, "q_out is NULL or not 16-byte aligned");
        if (n_q_heads < 1 || n_q_heads > c->cfg.max_q_heads) return fail(KVQ_EINVAL, "n_q_heads outside [1, max_q_heads]");
        const long long qd = (long long)n_q_heads * c->cfg.head_dim;
        if ((st = check_stride("q", q, q_stride, qd)) != KVQ_OK) return st;
        if (q_out == q && q_stride != qd) return fail(KVQ_EINVAL, "q is rotated in place only when it is dense");
    }
    a.g = c->g;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.Hq = n_q_heads;
    a.bf16 = dtype == KVQ_BF16;
    a.rope_dim = c->cfg.rope_dim;
    a.interleaved = c->cfg.rope_interleaved;
    // one row a sequence: the warp that stores it renews its page's bounds
    const bool one = !starts && T == 1;
    if (c->cfg.bounds && one) {
        a.codes = c->codes;
        a.scales = c->scales;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_append(a, c->freqs, c->num_sms, s);
    if (e != cudaSuccess) return cuda_fail(e, "paged append kernel");
    return c->cfg.bounds && !one ? bounds_of(c, a.r, s) : KVQ_OK;
}

kvq_status kvq_paged_read(kvq_paged* c, void* k_out, void* v_out, kvq_dtype dtype, const int* tables, const int* lens,
                          int n_seq, int T, const int* starts, int rows, void* stream) {
    if (!c) return fail(KVQ_EINVAL, "cache is NULL");
    if (dtype != KVQ_F32 && dtype != KVQ_BF16) return fail(KVQ_EINVAL, "dtype must be f32 or bf16");
    ReadArgs a = {};
    kvq_status st = check_rows(c, tables, lens, n_seq, T, starts, rows, &a.r);
    if (st != KVQ_OK || rows == 0) return st;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
        return fail(KVQ_EINVAL, "k_out or v_out is NULL or not 16-byte aligned");
    a.g = c->g;
    a.k_out = k_out;
    a.v_out = v_out;
    a.bf16 = dtype == KVQ_BF16;
    cudaError_t e = launch_read(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVQ_OK : cuda_fail(e, "paged read kernel");
}

kvq_status kvq_paged_bounds(kvq_paged* c, const int* tables, const int* lens, int n_seq, int T, const int* starts,
                            int rows, void* stream) {
    if (!c) return fail(KVQ_EINVAL, "cache is NULL");
    if (!c->cfg.bounds) return fail(KVQ_EINVAL, "the cache keeps no bounds (config.bounds)");
    Rows r;
    kvq_status st = check_rows(c, tables, lens, n_seq, T, starts, rows, &r);
    if (st != KVQ_OK || rows == 0) return st;
    return bounds_of(c, r, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_paged_decode(kvq_paged* c, const kvq_paged_query* a, void* stream) {
    return decode(c, a, nullptr, nullptr, 0, nullptr, 0, stream);
}

kvq_status kvq_paged_decode_shared(kvq_paged* c, const kvq_paged_query* a, const int* group_start,
                                   const int* prefix_len, int n_groups, void* stream) {
    kvq_status st = check_query(c, a);
    if (st != KVQ_OK) return st;
    if (!group_start || !prefix_len) return fail(KVQ_EINVAL, "group_start or prefix_len is NULL");
    if (n_groups < 1 || n_groups > a->n_seq) return fail(KVQ_EINVAL, "n_groups must be in [1, n_seq]");
    return decode(c, a, group_start, prefix_len, n_groups, nullptr, 0, stream);
}

kvq_status kvq_paged_select(kvq_paged* c, const kvq_paged_query* a, int* pages, int keep, int n_first, int n_last,
                            void* stream) {
    kvq_status st = check_query(c, a);
    if (st != KVQ_OK) return st;
    if (!c->cfg.bounds) return fail(KVQ_EINVAL, "the cache keeps no bounds (config.bounds)");
    if (!pages) return fail(KVQ_EINVAL, "pages is NULL");
    if (a->n_seq * a->T > kMaxEntries) return fail(KVQ_ERANGE, "n_seq * T above %d", kMaxEntries);
    if (n_first < 0 || n_last < 0 || keep < 1 || n_first > keep || n_last > keep - n_first)
        return fail(KVQ_EINVAL, "keep must be >= 1 and hold n_first + n_last pages");
    SelectArgs s = {};
    s.g = c->g;
    s.codes = c->codes;
    s.scales = c->scales;
    s.q = a->q;
    s.bf16 = a->dtype == KVQ_BF16;
    s.n_seq = a->n_seq;
    s.T = a->T;
    s.Hq = a->n_q_heads;
    s.hpk = a->n_q_heads / c->cfg.n_kv_heads;
    s.tables = a->tables;
    s.lens = a->lens;
    s.pages = pages;
    s.keys = reinterpret_cast<uint32_t*>(c->ws + c->off_keys);
    s.arrived = reinterpret_cast<int*>(c->ws + c->off_arrived);
    s.key_stride = (int)round_up(c->cfg.max_pages, 4);
    s.keep = keep;
    s.n_first = n_first;
    s.n_last = n_last;
    cudaError_t e = launch_select(s, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVQ_OK : cuda_fail(e, "page selection kernel");
}

kvq_status kvq_paged_decode_sparse(kvq_paged* c, const kvq_paged_query* a, const int* pages, int keep, void* stream) {
    kvq_status st = check_query(c, a);
    if (st != KVQ_OK) return st;
    if (!pages || keep < 1) return fail(KVQ_EINVAL, "pages is NULL or keep below 1");
    if ((long long)keep * c->cfg.page_rows > (1LL << 24)) return fail(KVQ_EINVAL, "keep * page_rows above 2^24");
    if (a->window != 0) return fail(KVQ_EINVAL, "listed pages take no window");
    if (a->n_seq * a->T > kMaxEntries) return fail(KVQ_ERANGE, "n_seq * T above %d", kMaxEntries);
    return decode(c, a, nullptr, nullptr, 0, pages, keep, stream);
}

kvq_status kvq_paged_read_error(kvq_paged* c, int* err, void* stream) {
    if (!c || !err) return fail(KVQ_EINVAL, "NULL argument");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // in the stream's own order: on another stream the clearing could fall behind the
    // next call's report
    int word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, c->g.err, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return cuda_fail(e, "read error word");
    e = cudaMemsetAsync(c->g.err, 0, sizeof(int), s);
    if (e != cudaSuccess) return cuda_fail(e, "clear error word");
    e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    *err = word;
    return KVQ_OK;
}

}  // extern "C"
