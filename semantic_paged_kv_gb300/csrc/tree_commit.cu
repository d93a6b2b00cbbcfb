// The accepted nodes' keys and values into the 4-bit caches of all layers:
// ice_cache4_commit.  Row path[b, i] of K and V goes to cache token start[b] +
// i in 4 bits (step, mid and codes as in ice.h).
//
// Eight lanes a row, four rows a warp at a time; a CTA stays with one (layer,
// sequence) and walks its rows, so that the few accepted ones of a wide tree
// cost no empty CTAs.
//
// Bound by the chain count - path - page number - row - codes, with one row of a lane group on its way at a time (issue 58% busy,
// DRAM 13% where there are many rows).  Measured: 32 layers of one sequence, 8 KV heads 2.8 us on the GPU (fp32 3.0), 64 layers of
// 16 sequences 11.5 us (fp32 11.6); their bytes take 0.1 and 3.6.
#include "common.cuh"
#include "internal.h"
#include "quant4.cuh"

namespace ice {
namespace {

constexpr int kThreads = 256, kRowsAtOnce = kThreads / 8;

struct CommitArgs {
    ice_rows k, v;
    long long k_layer, v_layer, records_layer;
    const int32_t *path, *n_path, *start;
    unsigned char *records;
    const int32_t *table;
    int n_pages, max_pages, hkv, n_nodes, batch, parts;
    int32_t *err;
};

template <typename T> __global__ void __launch_bounds__(kThreads) k_cache4_commit(const __grid_constant__ CommitArgs A) {
    const int l = threadIdx.x & 7;
    const int part = blockIdx.x % A.parts, lb = blockIdx.x / A.parts;
    const int b = lb % A.batch, layer = lb / A.batch;
    dep_wait();
    const int n = min(max(A.n_path[b], 0), A.n_nodes), start = A.start[b];
    unsigned char *records = A.records + (long long)layer * A.records_layer;
    const long long rows = 2ll * n * A.hkv;  // (node of the path, K or V, head)
    for (long long r0 = (long long)part * kRowsAtOnce; r0 < rows; r0 += (long long)A.parts * kRowsAtOnce) {
        const long long r = r0 + (threadIdx.x >> 3);
        bool live = r < rows;
        q4::Vec8<T> x, y;
        x.zero(), y.zero();
        int h = 0, kv = 0;
        unsigned char *rec = nullptr;
        int slot = 0;
        if (live) {
            const int i = (int)(r / (2 * A.hkv)), rest = (int)(r % (2 * A.hkv));
            kv = rest / A.hkv, h = rest % A.hkv;
            const int node = A.path[(long long)b * A.n_nodes + i];
            const long long at = (long long)start + i;
            live = node >= 0 && node < A.n_nodes && at >= 0 && at < (long long)A.max_pages * kPage;
            int page = -1;
            if (live) page = A.table[(long long)b * A.max_pages + at / kPage];
            live = live && page >= 0 && page < A.n_pages;
            if (live) {
                const ice_rows &v = kv ? A.v : A.k;
                const T *src = static_cast<const T *>(v.data) + (long long)layer * (kv ? A.v_layer : A.k_layer) +
                               (long long)b * v.batch + (long long)node * v.token + (long long)h * v.head;
                x.load(src + l * 8);
                y.load(src + 64 + l * 8);
                rec = records + ((long long)page * A.hkv + h) * q4::kRecord;
                slot = (int)(at % kPage);
            } else if (l == 0) {
                set_err(A.err, ICE_ERR_CAPACITY);
            }
        }
        uint32_t cx, cy;
        uint2 meta;
        q4::quantise_row<T>(x, y, l, l + 8, live, cx, cy, meta);
        if (!live) continue;
        if (kv)
            q4::put_v(rec, slot, l, l + 8, cx, cy);
        else
            q4::put_k(rec, slot, l, l + 8, cx, cy);
        if (l == 0) *reinterpret_cast<uint2 *>(rec + (kv ? q4::kVMeta : q4::kKMeta) + slot * 8) = meta;
    }
}

}  // namespace

cudaError_t launch_cache4_commit(const ice_params &p, int n_layers, int n_nodes, const ice_rows &k, const ice_rows &v,
                                 long long k_layer, long long v_layer, const int32_t *path, const int32_t *n_path,
                                 const int32_t *start, const ice_cache4 &cache, long long records_layer, int32_t *err,
                                 cudaStream_t s) {
    CommitArgs A{};
    A.k = k, A.v = v, A.k_layer = k_layer, A.v_layer = v_layer, A.records_layer = records_layer;
    A.path = path, A.n_path = n_path, A.start = start;
    A.records = static_cast<unsigned char *>(cache.records);
    A.table = cache.table, A.n_pages = cache.n_pages, A.max_pages = cache.max_pages;
    A.hkv = p.n_kv_heads, A.n_nodes = n_nodes, A.batch = p.batch, A.err = err;
    // CTAs of one (layer, sequence): as many as its rows can use, while all of them fit the GPU about once
    const long long lb = (long long)n_layers * p.batch;
    const int want = ceil_div(2ll * n_nodes * p.n_kv_heads, kRowsAtOnce), room = (int)(8 * device_sms() / lb);
    A.parts = want < 1 ? 1 : (want < room ? want : (room < 1 ? 1 : room));
    auto kern = p.dtype == ICE_BF16 ? k_cache4_commit<__nv_bfloat16> : k_cache4_commit<float>;
    return launch_dependent(kern, dim3((unsigned)(lb * A.parts)), dim3(kThreads), 0, s, A);
}

}  // namespace ice
