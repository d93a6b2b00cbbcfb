// Attention of drafted tokens over 4-bit pages: what its kernels share -- the
// cut of the work into runs, the ancestors of nodes, and partial results.
//
// A unit (sequence, KV head) with n nodes has n g query rows (row r: node r / g,
// head r % g of the group), cut into blocks of R rows.  A segment is one block
// and all that it attends to: tiles of 8 pages (128 slots; selected pages, then
// the cache's), then tiles of 128 nodes up to the block's last one.  The tiles
// of all segments, one after another, are cut into equal runs, one per CTA,
// whatever the lengths; a segment counts kTreeOver tiles more than it has (what
// starting and ending one costs).  A segment that runs cut leaves partial
// results in the workspace, joined in a fixed order by a second kernel.  Where every
// segment has a CTA and none is much longer than such a run, all stay whole.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "quant4.cuh"

namespace ice {
namespace tree {

constexpr int kTile = 128;                  // slots or nodes of a tile
constexpr int kTilePages = kTile / kPage;
constexpr int kMaxNodes = ICE_TREE_NODES;   // of a tree with parents
constexpr int kWords = kMaxNodes / 32;
constexpr int kPartRows = 128;              // rows of a partial result, at most
// Tiles that a segment takes beside its own (queries, ancestors, results), by the rows of a block.  128 rows: 9 ragged
// sequences of 32 heads and four sets of lengths take 75, 50, 51 and 151 us with 4, 70, 50, 52 and 134 with 5, 67, 49, 50 and 124
// with 6, 69, 49, 55 and 108 with 8; one tree at 16k 27.4 with 4, 28.2 with 6, 27.8 with 8.
template <int R> constexpr int kTreeOver = R == 128 ? 6 : 1;
// Places by which the longest segment may pass an equal run so that, where there is a CTA for each and they fill a quarter of the
// CTAs, all stay whole: a cut costs another start and end, and the join.  128 rows, whole and cut: 26 places against equal runs
// of 22 40 and 49 us, of 17 40 and 40 (of different lengths 40 and 50), of 11 39 and 34; 15 against 13 25 and 34, against 7 27
// and 29, against 4 24 and 19; 74 against 63 103 and 86; 8 segments of 10 against 1 21 and 19.
template <int R> constexpr int kTreeWhole = R == 128 ? 9 : 1;
constexpr int kMinRun = 1;  // places of a run, at least (the tiny fp32 layout takes 48 us with 2, 29 with 1)

// The segment that starts in a CTA and goes on in the next ones (runs 0: none).
struct Part {
    int32_t unit, block, rows;
    int16_t runs, inside;
};

struct Args {
    ice_rows q, k, v, o;
    const int32_t *parents, *counts;
    int n_nodes;
    const unsigned char *pool;  // selected pages (NULL: none)
    const int32_t *page_len, *sel_pages, *sel_count;
    int page_cap, max_sel;
    const unsigned char *cache;  // token-ordered pages (NULL: none)
    const int32_t *table, *lens;
    int n_pages, max_pages;
    int g, hq, hkv, units;
    float scale;
    float4 *part_o;   // [2 CTAs, 32, kPartRows]: elements 4 i .. of a row's result over the run's tokens
    float2 *part_ml;  // [2 CTAs, kPartRows]: its maximum (powers of two) and sum (times any number, the same for all)
    Part *parts;      // [CTAs]
    int32_t *err;
    int fault;  // ICE_FAULT's timeout: the kernel's producers deliver no values
};

__device__ __forceinline__ int nodes_of(const Args &A, int b) {
    return A.counts ? min(max(A.counts[b], 0), A.n_nodes) : A.n_nodes;
}
// (selected pages, cache tokens) of a unit.
__device__ __forceinline__ int2 counts_of(const Args &A, int u) {
    int2 n = make_int2(0, 0);
    if (A.pool) n.x = min(max(A.sel_count[u], 0), A.max_sel);
    if (A.cache) {
        const int t = A.lens[u / A.hkv], most = A.max_pages * kPage;  // < 2^31
        if (t < 0 || t > most) set_err(A.err, ICE_ERR_CAPACITY);
        n.y = min(max(t, 0), most);
    }
    return n;
}
__device__ __forceinline__ int pages_of(int2 n) { return n.x + (n.y + kPage - 1) / kPage; }
// (pages < 2^28: no overflow)
__device__ __forceinline__ int page_tiles(int2 n) { return (pages_of(n) + kTilePages - 1) / kTilePages; }

// Unit u, block blk: its tiles start at place `first` of the run (a negative
// one before it), n of them, the first n_page of pages.
struct Segment {
    int u, blk, blocks, nodes;
    int2 cnt;
    int n_page, n;
    long long first;
    __device__ __forceinline__ long long end() const { return first + n; }
};

template <int R> __device__ __forceinline__ int node_tiles(int nodes, int g, int blk) {
    const int last = ((blk + 1) * R - 1) / g;  // (n_nodes g <= 2^30)
    return min(last, nodes - 1) / kTile + 1;
}
template <int R> __device__ __forceinline__ int blocks_of(int nodes, int g) {
    return (nodes * g + R - 1) / R;
}
// Segments (2^20 at most are counted), their places and those of the longest one.
struct Load {
    long long places;
    int segments, most;
};
template <int R> __device__ __forceinline__ void add_unit(int2 cnt, int nodes, int g, Load &l) {
    const int blocks = blocks_of<R>(nodes, g), each = page_tiles(cnt) + kTreeOver<R>;
    for (int i = 0; i < blocks; ++i) {
        const int n = each + node_tiles<R>(nodes, g, i);
        l.places += n, l.most = max(l.most, n);
    }
    l.segments = min(l.segments + blocks, 1 << 20);
}
template <int R> __device__ __forceinline__ void load_unit(const Args &A, int u, Segment &s) {
    s.u = u;
    s.blk = 0;
    s.nodes = nodes_of(A, u / A.hkv);
    s.cnt = counts_of(A, u);
    s.blocks = blocks_of<R>(s.nodes, A.g);
    s.n_page = page_tiles(s.cnt);
}
template <int R> __device__ __forceinline__ void size_segment(const Args &A, long long place, Segment &s) {
    s.n = s.n_page + node_tiles<R>(s.nodes, A.g, s.blk);
    s.first = place + kTreeOver<R>;
}
// The segment after s.
template <int R> __device__ __forceinline__ void next_segment(const Args &A, Segment &s) {
    const long long place = s.end();
    if (++s.blk >= s.blocks) {
        int u = s.u;
        do load_unit<R>(A, ++u, s);
        while (s.blocks == 0 && u + 1 < A.units);
    }
    size_segment<R>(A, place, s);
}

struct PlanScratch {
    Load sum[32];
    Segment seg;
    int n;
};
struct Run {
    long long f0, share;
    int n;  // places (0: none)
};
// This CTA's run and its first segment (all threads call; S is read by all after it returns).
template <int R, int kThreads> __device__ __forceinline__ Run plan_run(const Args &A, PlanScratch &S) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (A.units + kThreads - 1) / kThreads;
    const int ua = min(tid * per, A.units), ub = min(ua + per, A.units);
    Load mine{0, 0, 0};
    for (int u = ua; u < ub; ++u) add_unit<R>(counts_of(A, u), nodes_of(A, u / A.hkv), A.g, mine);
    long long before = mine.places;
    int segments = mine.segments;
    const int most_of_warp = __reduce_max_sync(0xffffffffu, mine.most);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, off);
        const int z = __shfl_up_sync(0xffffffffu, segments, off);
        if (lane >= off) before += y, segments += z;
    }
    if (lane == 31) S.sum[warp] = Load{before, segments, most_of_warp};
    __syncthreads();
    Load all{0, 0, 0};
    before -= mine.places, segments -= mine.segments;
    const int warps = min(kThreads / 32, (A.units + 31) / 32);  // that have units
    for (int w = 0; w < warps; ++w) {
        const Load x = S.sum[w];
        if (w < warp) before += x.places, segments += x.segments;
        all.places += x.places, all.segments += x.segments, all.most = max(all.most, x.most);
    }
    const long long total = all.places;
    Run r;
    r.share = total < (1ll << 30) ? ((unsigned)total + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
    if (r.share < kMinRun) r.share = kMinRun;
    const bool whole = all.segments <= (int)gridDim.x && 4 * all.segments > (int)gridDim.x && all.most <= r.share + kTreeWhole<R>;
    r.f0 = r.share * blockIdx.x;
    r.n = (int)max(min(r.share, total - r.f0), 0ll);
    if (whole) r.n = (int)blockIdx.x < all.segments;
    if (whole ? (int)blockIdx.x >= segments && (int)blockIdx.x < segments + mine.segments
              : r.n > 0 && r.f0 >= before && r.f0 < before + mine.places) {
        long long at = before;
        for (int u = ua; u < ub; ++u) {
            Segment s;
            load_unit<R>(A, u, s);
            for (; s.blk < s.blocks; ++s.blk, ++segments) {
                size_segment<R>(A, whole ? 0 : at - r.f0, s);
                if (whole ? segments == (int)blockIdx.x : s.end() > 0) break;
                at = s.end() + r.f0;
            }
            if (s.blk < s.blocks) {
                S.seg = s;
                S.n = (int)s.end();
                break;
            }
        }
    }
    __syncthreads();
    if (whole && r.n) r.n = S.n;
    return r;
}
// A segment whose first tile is in this CTA's run (a full one) and whose last one is not: its runs.  (One at most starts in
// a CTA.)
template <int R> __device__ __forceinline__ Part part_of(const Segment &s, const Run &r, int g) {
    const long long beyond = s.end() - r.n;
    const int more = beyond < (1ll << 30) && r.share < (1ll << 30)
                         ? (int)(((unsigned)beyond + (unsigned)r.share - 1) / (unsigned)r.share)
                         : (int)((beyond + r.share - 1) / r.share);
    return Part{s.u, s.blk, min(R, s.nodes * g - s.blk * R), (int16_t)(1 + more), (int16_t)(s.first > 0 ? 1 : 0)};
}

// Ancestors of the nodes of a tree, themselves among them, by pointer jumping.
struct Ancestors {
    uint32_t mask[kMaxNodes][kWords];
    int16_t up[kMaxNodes];
};
// By kMaxNodes threads, thread t node t with parent `up`, with a barrier among them as `sync`.
template <typename Sync>
__device__ __forceinline__ void find_ancestors(int up, int nodes, Ancestors &X, int32_t *err, int t, Sync sync) {
    uint32_t mine[kWords];
    if (t < nodes && (up >= t || up < -1)) {
        set_err(err, ICE_ERR_INVALID_ARG);
        up = -1;
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) mine[w] = w == t >> 5 ? 1u << (t & 31) : 0u;
    for (int reach = 1;; reach <<= 1) {
        if (t < nodes) {
            X.up[t] = (int16_t)up;
#pragma unroll
            for (int w = 0; w < kWords; ++w) X.mask[t][w] = mine[w];
        }
        sync();
        if (reach >= nodes) return;
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) mine[w] |= X.mask[up][w];
            up = X.up[up];
        }
        sync();
    }
}

// Record and used slots of a unit's page x, whose number is id (nullptr: there is no such page).
__device__ __forceinline__ const unsigned char *page_of_id(const Args &A, int u, int2 cnt, int x, int id, int &len) {
    len = 0;
    if (x < cnt.x) {
        if (id >= 0 && id < A.page_cap) {
            const size_t at = (size_t)u * A.page_cap + id;
            len = min(max(A.page_len[at], 0), kPage);
            return A.pool + at * q4::kRecord;
        }
    } else if (id >= 0 && id < A.n_pages) {
        const int b = u / A.hkv;
        len = min(cnt.y - (x - cnt.x) * kPage, kPage);
        return A.cache + ((size_t)id * A.hkv + (u - b * A.hkv)) * q4::kRecord;
    }
    set_err(A.err, ICE_ERR_CAPACITY);
    return nullptr;
}
// (x < pages_of(cnt))
__device__ __forceinline__ const unsigned char *page_at(const Args &A, int u, int2 cnt, int x, int &len) {
    const int id = x < cnt.x ? A.sel_pages[(size_t)u * A.max_sel + x]
                             : A.table[(size_t)(u / A.hkv) * A.max_pages + (x - cnt.x)];
    return page_of_id(A, u, cnt, x, id, len);
}

// Place of elements 4 i .. of row r of a partial result.
__device__ __forceinline__ size_t part_at(size_t slot, int i, int r) {
    return (slot * (kHeadDim / 4) + i) * kPartRows + r;
}

template <typename T> __device__ __forceinline__ const T *row_ptr(const ice_rows &r, int b, int t, int h) {
    return static_cast<const T *>(r.data) + (long long)b * r.batch + (long long)t * r.token + (long long)h * r.head;
}
template <typename T> __device__ __forceinline__ T *row_out(const ice_rows &r, int b, int t, int h) {
    return static_cast<T *>(r.data) + (long long)b * r.batch + (long long)t * r.token + (long long)h * r.head;
}
// Four elements of a row, rounded to its type.
__device__ __forceinline__ void put4(float *out, float4 x) { *reinterpret_cast<float4 *>(out) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16 *out, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(out) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

}  // namespace tree

// The attention kernels: their runs' results, the cut segments' in parts (joined by launch_tree).
constexpr int kTreeRowsSimt = 64, kTreeRowsTc = 128;  // rows of a block
cudaError_t launch_tree_simt(const tree::Args &A, int grid, cudaStream_t s);
cudaError_t launch_tree_tc(const tree::Args &A, int grid, cudaStream_t s);

}  // namespace ice
