// Attention of drafted tokens over 4-bit pages: the launches of
// ice_cache4_attn_tree and ice_sparse_attn_tree4, and the join of what runs of
// work cut (a kernel of its own: with many runs a segment its rows keep the
// whole GPU busy, where a last CTA would join them alone).
#include <float.h>

#include <algorithm>

#include "tree.cuh"

namespace ice {
namespace {

using namespace tree;

// All CTAs find the cut segments in `parts` and take pieces of them in turn: 32 rows (neighbours in the parts) and either 32
// elements, 4 a warp, or, where a segment has more than kAhead runs, 8 elements, 4 a warp and a quarter of the runs.
// (One tree at 16k, 8 segments of 19 runs: about 4 us of the call; 7 with whole columns of runs a warp and CTAs for every place
// of `parts`.  What is left is the launch, the list and one or two passes through the memory's latency.)
constexpr int kJoinCtas = 4;  // an SM
constexpr int kMostParts = 256;
constexpr int kAhead = 5, kSplit = 4;
// Infinities and NaN of a part go to `odd`: they reach the result whatever the part weighs, as in a segment that is not cut.
__device__ __forceinline__ void set_apart(float &v, float &odd) {
    if (!(fabsf(v) < INFINITY)) odd += v, v = 0.f;
}
__device__ __forceinline__ void set_apart(float4 &v, float4 &odd) {
    if (fabsf(v.x) + fabsf(v.y) + (fabsf(v.z) + fabsf(v.w)) < INFINITY) return;
    set_apart(v.x, odd.x), set_apart(v.y, odd.y), set_apart(v.z, odd.z), set_apart(v.w, odd.w);
}
struct Cut {
    Part p;
    int run, first;  // its first run, the number of its first piece
};
template <typename T, int kBlock>
__global__ void __launch_bounds__(256, kJoinCtas) k_tree_join(const __grid_constant__ Args A, int n_parts) {
    constexpr int kGroups = kBlock / 32;
    __shared__ Cut cuts[kMostParts + 1];
    __shared__ int2 of_warp[8];  // cuts, pieces
    __shared__ float4 sum[kSplit][2][32];
    __shared__ float2 ml_of[kSplit][2][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto is_split = [](const Part &p) { return p.runs > kAhead; };
    dep_wait();
    int pieces, n_cuts;
    {
        Part p{};
        if (tid < n_parts) p = A.parts[tid];
        const int mine = p.runs == 0 ? 0 : kGroups * (is_split(p) ? kHeadDim / 8 : kHeadDim / 32);
        const unsigned hit = __ballot_sync(0xffffffffu, mine > 0);
        int before = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += y;
        }
        if (lane == 31) of_warp[warp] = make_int2(__popc(hit), before);
        __syncthreads();
        int at = __popc(hit & ((1u << lane) - 1u));
        before -= mine, pieces = 0, n_cuts = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const int2 x = of_warp[w];
            if (w < warp) at += x.x, before += x.y;
            n_cuts += x.x, pieces += x.y;
        }
        if (mine > 0) cuts[at] = Cut{p, tid, before};
        __syncthreads();
    }
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        int lo = 0, hi = n_cuts;  // the last cut that starts at or before this piece
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            (cuts[mid].first <= piece ? lo : hi) = mid;
        }
        const Cut &c = cuts[lo];
        const Part &p = c.p;
        const bool split = is_split(p);
        const int x = piece - c.first, r = x % kGroups * 32 + lane;
        const int i = split ? x / kGroups * 2 + (warp & 1) : x / kGroups * 8 + warp;  // 4 elements
        const int k_first = split ? warp >> 1 : 0, k_step = split ? kSplit : 1, runs = p.runs;
        const bool live = r < p.rows;
        float M = -FLT_MAX, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), odd = acc;
        for (int k0 = k_first; live && k0 < runs; k0 += kAhead * k_step) {
            float2 ml[kAhead];
            float4 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int k = k0 + j * k_step;
                ml[j] = make_float2(-FLT_MAX, 0.f), v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < runs) {
                    const size_t slot = (size_t)(2 * (c.run + k) + (k == 0 ? p.inside : 0));
                    ml[j] = A.part_ml[slot * kPartRows + r];
                    v[j] = A.part_o[part_at(slot, i, r)];
                }
            }
            float top = M;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) top = fmaxf(top, ml[j].x);
            const float f = exp2f(M - top);
            M = top;
            L *= f, acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                set_apart(v[j], odd);
                if (ml[j].y == 0.f) continue;
                const float w = ml[j].y * exp2f(ml[j].x - M);
                L += w;
                if (w != 0.f) {
                    acc.x = fmaf(v[j].x, w, acc.x), acc.y = fmaf(v[j].y, w, acc.y);
                    acc.z = fmaf(v[j].z, w, acc.z), acc.w = fmaf(v[j].w, w, acc.w);
                }
            }
        }
        if (split) {  // (the same for the whole CTA)
            acc.x += odd.x, acc.y += odd.y, acc.z += odd.z, acc.w += odd.w;
            sum[warp >> 1][warp & 1][lane] = acc, ml_of[warp >> 1][warp & 1][lane] = make_float2(M, L);
            __syncthreads();
            if (warp < 2) {
#pragma unroll
                for (int k = 1; k < kSplit; ++k) M = fmaxf(M, ml_of[k][warp][lane].x);
                acc = odd = make_float4(0.f, 0.f, 0.f, 0.f), L = 0.f;
#pragma unroll
                for (int k = 0; k < kSplit; ++k) {
                    const float2 ml = ml_of[k][warp][lane];
                    float4 v = sum[k][warp][lane];
                    set_apart(v, odd);
                    if (ml.y == 0.f) continue;
                    const float f = exp2f(ml.x - M);
                    L = fmaf(ml.y, f, L);
                    acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
                }
            }
            __syncthreads();
        }
        if (live && (!split || warp < 2)) {
            const int b = p.unit / A.hkv, h = p.unit - b * A.hkv, row = p.block * kBlock + r;
            const float inv = 1.f / L;
            put4(row_out<T>(A.o, b, row / A.g, h * A.g + row % A.g) + 4 * i,
                 make_float4(fmaf(acc.x, inv, odd.x), fmaf(acc.y, inv, odd.y), fmaf(acc.z, inv, odd.z),
                             fmaf(acc.w, inv, odd.w)));
        }
    }
}

struct Ws {
    float4 *part_o;
    float2 *part_ml;
    Part *parts;
    size_t bytes;
};
Ws ws_layout(int ctas, void *base) {
    Ws w{};
    char *b = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *r = b ? b + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return r;
    };
    w.part_o = reinterpret_cast<float4 *>(take(sizeof(float) * 2 * ctas * kPartRows * kHeadDim));
    w.part_ml = reinterpret_cast<float2 *>(take(sizeof(float2) * 2 * ctas * kPartRows));
    w.parts = reinterpret_cast<Part *>(take(sizeof(Part) * ctas));
    w.bytes = off;
    return w;
}
static_assert(kTreeRowsSimt <= kPartRows && kTreeRowsTc <= kPartRows, "rows of a partial result");

template <typename T, int kBlock> cudaError_t launch_join(const Args &A, int grid, cudaStream_t s) {
    return launch_dependent(k_tree_join<T, kBlock>, dim3(kJoinCtas * device_sms()), dim3(256), 0, s, A, grid);
}

}  // namespace

double tree_tiles(const ice_params &p, int n_nodes, double pages) {
    const double rows = (double)n_nodes * (p.n_q_heads / p.n_kv_heads), blocks = rows / kTreeRowsSimt + 1;
    return units_of(p) * blocks * (pages / kTilePages + n_nodes / kTile + 8);
}

static int grid_of() { return std::min(device_sms(), kMostParts); }  // one CTA an SM
size_t tree_workspace() { return ws_layout(grid_of(), nullptr).bytes; }

cudaError_t launch_tree(const ice_params &p, const ice_tree &t, const ice_rows &q, const void *records,
                        const int32_t *page_len, const int32_t *sel_pages, const int32_t *sel_count, int max_sel,
                        const ice_cache4 *cache, const int32_t *lens, const ice_rows &k, const ice_rows &v, float scale,
                        const ice_rows &o, void *ws, int32_t *err, cudaStream_t s) {
    Args A{};
    A.q = q, A.k = k, A.v = v, A.o = o;
    A.parents = t.parents, A.counts = t.counts, A.n_nodes = t.n_nodes;
    A.pool = static_cast<const unsigned char *>(records);
    A.page_len = page_len, A.sel_pages = sel_pages, A.sel_count = sel_count;
    A.page_cap = p.page_cap, A.max_sel = max_sel;
    if (cache) {
        A.cache = static_cast<const unsigned char *>(cache->records);
        A.table = cache->table, A.n_pages = cache->n_pages, A.max_pages = cache->max_pages;
        A.lens = lens;
    }
    A.g = p.n_q_heads / p.n_kv_heads, A.hq = p.n_q_heads, A.hkv = p.n_kv_heads, A.units = units_of(p);
    A.scale = scale;
    A.err = err;
    A.fault = fault_armed("timeout");
    const int grid = grid_of();
    const Ws w = ws_layout(grid, ws);
    A.part_o = w.part_o, A.part_ml = w.part_ml, A.parts = w.parts;
    if (p.dtype == ICE_BF16) {
        const cudaError_t e = launch_tree_tc(A, grid, s);
        return e != cudaSuccess ? e : launch_join<__nv_bfloat16, kTreeRowsTc>(A, grid, s);
    }
    const cudaError_t e = launch_tree_simt(A, grid, s);
    return e != cudaSuccess ? e : launch_join<float, kTreeRowsSimt>(A, grid, s);
}

}  // namespace ice
