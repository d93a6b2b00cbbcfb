// Attention of drafted tokens over 4-bit pages: the launches of
// ice_cache4_attn_tree and ice_sparse_attn_tree4, and the join of what runs of
// work cut (a kernel of its own: with many runs a segment its rows keep the
// whole GPU busy, where a last CTA would join them alone).
#include <float.h>

#include "tree.cuh"

namespace ice {
namespace {

using namespace tree;

// CTA (c, y) joins rows 32 (y % (kBlock / 32)) .. and elements 32 (y / (kBlock / 32)) .. of the segment that starts in
// run c: a warp takes 32 rows (neighbours in the parts) and 4 elements.
template <typename T, int kBlock>
__global__ void __launch_bounds__(256) k_tree_join(const __grid_constant__ Args A) {
    constexpr int kGroups = kBlock / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
    dep_wait();
    const Part p = A.parts[c];
    if (p.runs == 0) return;
    const int b = p.unit / A.hkv, h = p.unit - b * A.hkv, nodes = nodes_of(A, b);
    const int row0 = p.block * kBlock, r = blockIdx.y % kGroups * 32 + lane, i = blockIdx.y / kGroups * 8 + warp;
    if (r >= min((long long)kBlock, (long long)nodes * A.g - row0)) return;
    auto slot_of = [&](int k) { return (size_t)(2 * (c + k) + (k == 0 ? p.inside : 0)); };
    // eight runs at a time, against the running maximum
    float M = -FLT_MAX, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < p.runs; k0 += 8) {
        float2 ml[8];
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ml[k] = make_float2(-FLT_MAX, 0.f);
            if (k0 + k < p.runs) {
                ml[k] = A.part_ml[slot_of(k0 + k) * kPartRows + r];
                x[k] = A.part_o[part_at(slot_of(k0 + k), i, r)];
            }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
        const float f = exp2f(M - top);
        M = top;
        L *= f, acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (ml[k].y == 0.f) continue;
            const float w = ml[k].y * exp2f(ml[k].x - M);
            L += w;
            if (w != 0.f) {
                acc.x = fmaf(x[k].x, w, acc.x), acc.y = fmaf(x[k].y, w, acc.y);
                acc.z = fmaf(x[k].z, w, acc.z), acc.w = fmaf(x[k].w, w, acc.w);
            }
        }
    }
    const float inv = 1.f / L;
    put4(row_out<T>(A.o, b, (row0 + r) / A.g, h * A.g + (row0 + r) % A.g) + 4 * i,
         make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
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
    return launch_dependent(k_tree_join<T, kBlock>, dim3(grid, kBlock / 32 * 4), dim3(256), 0, s, A);
}

}  // namespace

double tree_tiles(const ice_params &p, int n_nodes, double pages) {
    const double rows = (double)n_nodes * (p.n_q_heads / p.n_kv_heads), blocks = rows / kTreeRowsSimt + 1;
    return units_of(p) * blocks * (pages / kTilePages + n_nodes / kTile + 8);
}

size_t tree_workspace() { return ws_layout(device_sms(), nullptr).bytes; }

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
    const int grid = device_sms();  // one CTA an SM
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
