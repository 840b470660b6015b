// Declarations shared by the paged-cache translation units: geometry, the cell
// layout (include/kvq.h), parameter blocks and launchers.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {
namespace paged {

constexpr int kCellRows = 16;
constexpr int kMaxFreq = 128;          // rope_dim / 2 at most
constexpr int kMaxSeqs = 1024;
constexpr int kMaxEntries = 2048;      // work entries of one decode

struct Geom {
    uint8_t* pool;
    int* err;
    int n_pages, page_rows, page_shift, max_pages;
    int Hkv, D, fp8;
    int cell_bytes;
    long long page_bytes;
    __host__ __device__ int NB() const { return D / 32; }
    __host__ __device__ int cells_per_page() const { return page_rows / kCellRows; }
};

// Rows of the batch entries: uniform (T each) or packed by starts
struct Rows {
    const int* tables;
    const int* lens;
    const int* starts;
    int n_seq, T, rows;
};

// Where a packed row lies: the byte of its cell for KV head 0 (heads are
// cells_per_page() cells apart) and its row in the cell; cell < 0: nowhere.
struct Place {
    long long cell;
    int pos, t;
    int first;             // position of the entry's first row of this call
    int len;
};

#ifdef __CUDACC__
// Launch as a programmatic dependent: the kernel waits (griddepcontrol.wait)
// before it reads anything, so its start overlaps the end of the one before
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Byte of a page for a position of a sequence, or -1 with the error word set
__device__ __forceinline__ long long page_at(const Geom& g, const int* table, int pos) {
    const int pg = table[pos >> g.page_shift];
    if (pg < 0 || pg >= g.n_pages) {
        atomicExch(g.err, kErrCounter);
        return -1;
    }
    return pg * g.page_bytes;
}

// Place of a row of entry i (i < 0: the row is none's)
__device__ __forceinline__ Place place_in(const Geom& g, const Rows& r, int row, int i, bool short_is_error) {
    Place p{-1, -1, 0, 0, 0};
    if (i < 0) return p;
    const int from = r.starts ? r.starts[i] : i * r.T, at = row - from;
    const int n = r.starts ? r.starts[i + 1] - from : r.T;
    p.len = r.lens[i];
    if (p.len < 0 || p.len > (long long)g.max_pages << g.page_shift || (short_is_error && p.len < n)) {
        atomicExch(g.err, kErrCounter);
        p.pos = -2;
        return p;
    }
    p.first = max(p.len - n, 0);
    p.pos = p.len - n + at;
    if (p.pos < 0) return p;
    const long long pg = page_at(g, r.tables + (long long)i * g.max_pages, p.pos);
    if (pg < 0) return p;
    p.cell = pg + (long long)((p.pos & (g.page_rows - 1)) >> 4) * g.cell_bytes;
    p.t = p.pos & 15;
    return p;
}

// Entry of a row: the last that starts at or before it, -1 outside them
__device__ __forceinline__ int entry_of_row(const Rows& r, int row) {
    if (!r.starts) return row / r.T;
    if (row < r.starts[0] || row >= r.starts[r.n_seq]) return -1;
    int lo = 0, hi = r.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (r.starts[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The same for rows row0 + lane, lane < W, by a warp: 32 starts a step, where the
// search of one row is a chain of loads
template <int W>
__device__ __forceinline__ int entry_of_rows(const Rows& r, int row0, int lane) {
    const int row = row0 + lane;
    if (!r.starts) return row / r.T;
    int i = -1;
    for (int c = 0; c < r.n_seq; c += 32) {
        const int st = c + lane < r.n_seq ? r.starts[c + lane] : 0x7fffffff;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int k = __popc(__ballot_sync(0xffffffffu, st <= row0 + w));
            if (lane == w) i += k;
        }
    }
    // (behind the last start, or starts in no order)
    if (i >= 0 && (r.starts[i] > row || r.starts[i + 1] <= row)) i = entry_of_row(r, row);
    return i;
}

__device__ __forceinline__ Place place_row(const Geom& g, const Rows& r, int row, bool short_is_error) {
    return place_in(g, r, row, entry_of_row(r, row), short_is_error);
}
#endif

// Rotation frequencies in turns per position, as a sum of two floats
struct Freqs {
    float2 f[kMaxFreq];
};

struct AppendArgs {
    Geom g;
    Rows r;
    const void* k;
    const void* v;
    const void* q;
    void* q_out;
    long long k_stride, v_stride, q_stride;
    int Hq, bf16, rope_dim, interleaved;
    int8_t* codes;         // bounds of the pages that one row each goes to, or NULL
    float* scales;
};
cudaError_t launch_append(const AppendArgs& a, const Freqs& f, int num_sms, cudaStream_t s);

struct ReadArgs {
    Geom g;
    Rows r;
    void* k_out;
    void* v_out;
    int bf16;
};
cudaError_t launch_read(const ReadArgs& a, cudaStream_t s);

struct BoundsArgs {
    Geom g;
    Rows r;
    int8_t* codes;         // [n_pages][Hkv][NB][2][32]
    float* scales;         // [n_pages][Hkv][NB]
};
cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t s);

struct SelectArgs {
    Geom g;
    const int8_t* codes;
    const float* scales;
    const void* q;
    int bf16, n_seq, T, Hq, hpk;
    const int* tables;
    const int* lens;
    int* pages;            // [n_seq][T][Hkv][keep]
    uint32_t* keys;        // [n_seq][T][Hkv][key_stride] scores as ordered integers
    int key_stride;        // max_pages in whole fours
    int* arrived;          // [n_seq * T * Hkv] CTAs done; 0 between calls
    int keep, n_first, n_last;
};
cudaError_t launch_select(const SelectArgs& a, cudaStream_t s);

struct PlanEntry;

// Decode.  Work entries: sequences (dense), sequences then prefix groups
// (shared), or (sequence, query row) pairs (sparse).  An entry has nc cells,
// nq queries per KV head taken in slices of `tile`, and its work is (nc + setup) *
// slices * Hkv; the total is cut into equal ranges, one for each group of warps of
// each CTA.  The part of a range inside one (entry, KV head, slice) key is a
// fragment and writes its record to slot range + key.
struct SplitArgs {
    Geom g;
    const void* q;
    void* out;
    int bf16;
    int n_seq, T, Hq, hpk;
    const int* tables;
    const int* lens;
    const float* sinks;
    float qscale;                  // scale * log2(e)
    float softcap_a, softcap_b;    // log2 units: s -> b * tanh(a * s); b == 0: off
    int window;
    const int* group_start;        // shared: prefix groups
    const int* prefix_len;
    int n_groups;
    const int* lists;              // sparse: [n_seq][T][Hkv][keep]
    int keep;
    int E;                         // work entries
    int G;                         // CTAs of the split kernel
    int tile;                      // queries of a slice (QPI): 8, or 16 where a key has more (split_tile)
    int setup;                     // what starting a key costs, in cells
    int gw, groups;                // warps of a group, groups of a CTA of the split kernel
    int rec_rows;                  // query rows of a record: min(tile, most queries of a key)
    int fuse;                      // 1: the last CTA of a key joins its records (no merge kernel)
    int* arrived;                  // [key] records written; 0 between calls
    long long max_keys;            // keys that the record area holds beside the CTAs' own
    float* part_o;                 // [slot][rec_rows][D]
    float* part_ml;                // [slot][rec_rows][2]  (max in log2 units, sum)
    struct PlanEntry* plan;        // [E + 1], written by CTA 0 for the merge
    int tiles;                     // 1: groups with many queries go to the tile kernel
    int tile_rows;                 // queries of its blocks
    long long max_keys2;           // its keys that the record area holds
    uint16_t* part2_o;             // [CTA + key][tile_rows][D] fp16, times a power of two for each row
    float* part2_ml;               // [CTA + key][tile_rows][4]  (max, sum, what takes the power out again, -)
    struct PlanEntry* plan2;       // [n_groups + 1]
};
// Work before an entry ((cells + setup) x slices), keys before it (slices), its
// cells, the first of them and its queries per KV head; entry E holds the totals.
// Of a sequence (or one of its query rows): its length and the rows before `lo`
// that are its group's.  Of a prefix group: its rows and first member.
struct PlanEntry {
    long long work;
    int keys, nc, c0, nq, rows, lo;
};
int split_tile(int NB, bool bf16, int most_queries);
int split_warps(int NB, int tile);
cudaError_t launch_split(const SplitArgs& a, cudaStream_t s);
cudaError_t launch_merge(const SplitArgs& a, cudaStream_t s);
// prefixes of groups with many bf16 queries, 128-row tiles on tcgen05 (kvq_paged_prefix.cu)
int prefix_rows_of(int NB);                               // tile_rows
cudaError_t launch_prefix(const SplitArgs& a, cudaStream_t s);

}  // namespace paged
}  // namespace kvq
