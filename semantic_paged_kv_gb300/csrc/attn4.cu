// Attention of one query token over 4-bit pages: ice_cache4_attn_decode (a
// token-ordered cache) and ice_sparse_attn_decode4 (selected pages of a pool,
// then a cache's tokens, in one softmax).
//   O = sum_j exp(scale q . k_j) v_j / sum_j exp(scale q . k_j),
// papernotes.org "IceCache: Memory-Efficient KV-cache Management for
// Long-Sequence LLMs", 关键设计 1, over the unit's pages only.
//
// One CTA per unit, one warp per page at a time: two lanes a token for the
// scores (one group of 64 each), four elements a lane for the values.
#include "common.cuh"
#include "internal.h"
#include "quant4.cuh"

namespace ice {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxG = 16;

struct Attn4Args {
    const void *Q;
    const unsigned char *pool;  // selected pages (NULL: none)
    const int32_t *page_len, *sel_pages, *sel_count;
    int page_cap, max_sel;
    const unsigned char *cache;  // token-ordered pages (NULL: none)
    const int32_t *table, *lens;
    int n_pages, max_pages;
    int g, hq, hkv;
    float scale;
    float *O, *lse;
    int32_t *err;
};

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_attn4(const __grid_constant__ Attn4Args A) {
    __shared__ float s_q[kMaxG][kHeadDim];
    __shared__ float s_p[kWarps][kPage];
    __shared__ float s_ml[kWarps][kMaxG][2];
    extern __shared__ float s_o[];  // [kWarps][g][128]
    const int u = blockIdx.x, b = u / A.hkv, h = u % A.hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    dep_wait();
    const T *q = static_cast<const T *>(A.Q) + ((size_t)b * A.hq + (size_t)h * A.g) * kHeadDim;
    for (int i = threadIdx.x; i < A.g * kHeadDim; i += blockDim.x) s_q[i / kHeadDim][i % kHeadDim] = Elem<T>::load(q + i);
    __syncthreads();
    int n_sel = 0, n_tok = 0;
    if (A.pool) n_sel = min(max(A.sel_count[u], 0), A.max_sel);
    if (A.cache) {
        n_tok = A.lens[b];
        const long long most = (long long)A.max_pages * kPage;
        if ((n_tok < 0 || n_tok > most) && threadIdx.x == 0) set_err(A.err, ICE_ERR_CAPACITY);
        n_tok = (int)min((long long)max(n_tok, 0), most);
    }
    const int n = n_sel + (n_tok + kPage - 1) / kPage;
    float m[kMaxG], l[kMaxG], o[kMaxG][4];
#pragma unroll
    for (int i = 0; i < kMaxG; ++i) {
        m[i] = -INFINITY;
        l[i] = o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    for (int x = warp; x < n; x += kWarps) {
        const unsigned char *rec;
        int len;
        if (x < n_sel) {
            const int pg = A.sel_pages[(size_t)u * A.max_sel + x];
            if (pg < 0 || pg >= A.page_cap) {
                if (lane == 0) set_err(A.err, ICE_ERR_CAPACITY);
                continue;
            }
            len = min(A.page_len[(size_t)u * A.page_cap + pg], kPage);
            rec = A.pool + ((size_t)u * A.page_cap + pg) * q4::kRecord;
        } else {
            const int blk = x - n_sel;
            const int pg = A.table[(size_t)b * A.max_pages + blk];
            if (pg < 0 || pg >= A.n_pages) {
                if (lane == 0) set_err(A.err, ICE_ERR_CAPACITY);
                continue;
            }
            len = min(n_tok - blk * kPage, kPage);
            rec = A.cache + ((size_t)pg * A.hkv + h) * q4::kRecord;
        }
        if (len <= 0) continue;
        const int t = lane >> 1, gr = lane & 1;
        const float2 km = q4::unpack_meta(*reinterpret_cast<const uint32_t *>(rec + q4::kKMeta + t * 8 + gr * 4));
        float kv[64];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            float y[8];
            q4::values_of(q4::get_k(rec, t, gr * 8 + w), km, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) kv[w * 8 + e] = y[e];
        }
#pragma unroll
        for (int hh = 0; hh < kMaxG; ++hh) {
            if (hh >= A.g) break;
            float d = 0.f;
#pragma unroll
            for (int e = 0; e < 64; ++e) d = fmaf(kv[e], s_q[hh][gr * 64 + e], d);
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            const float s = t < len ? d * A.scale : -INFINITY;
            float mx = s;
#pragma unroll
            for (int off = 2; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m[hh], mx);
            const float al = m[hh] == -INFINITY ? 0.f : expf(m[hh] - mn);
            const float p = t < len ? expf(s - mn) : 0.f;
            float sum = p;
#pragma unroll
            for (int off = 2; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            m[hh] = mn;
            l[hh] = l[hh] * al + sum;
            __syncwarp();
            if (gr == 0) s_p[warp][t] = p;
            __syncwarp();
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int tt = 0; tt < len; ++tt) {
                const float2 vm =
                    q4::unpack_meta(*reinterpret_cast<const uint32_t *>(rec + q4::kVMeta + tt * 8 + (lane >> 4) * 4));
                const uint32_t c = *reinterpret_cast<const uint16_t *>(rec + q4::v_piece(tt, lane));
                const float pp = s_p[warp][tt];
                acc.x = fmaf(pp, fmaf(vm.x, (float)(c & 15u) - 7.5f, vm.y), acc.x);
                acc.y = fmaf(pp, fmaf(vm.x, (float)(c >> 4 & 15u) - 7.5f, vm.y), acc.y);
                acc.z = fmaf(pp, fmaf(vm.x, (float)(c >> 8 & 15u) - 7.5f, vm.y), acc.z);
                acc.w = fmaf(pp, fmaf(vm.x, (float)(c >> 12 & 15u) - 7.5f, vm.y), acc.w);
            }
            o[hh][0] = fmaf(o[hh][0], al, acc.x);
            o[hh][1] = fmaf(o[hh][1], al, acc.y);
            o[hh][2] = fmaf(o[hh][2], al, acc.z);
            o[hh][3] = fmaf(o[hh][3], al, acc.w);
        }
    }
#pragma unroll
    for (int hh = 0; hh < kMaxG; ++hh) {
        if (hh >= A.g) break;
        if (lane == 0) s_ml[warp][hh][0] = m[hh], s_ml[warp][hh][1] = l[hh];
#pragma unroll
        for (int e = 0; e < 4; ++e) s_o[((size_t)warp * A.g + hh) * kHeadDim + lane * 4 + e] = o[hh][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < A.g * kHeadDim; i += blockDim.x) {
        const int hh = i / kHeadDim;
        float M = -INFINITY, L = 0.f, acc = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][hh][0]);
        for (int w = 0; w < kWarps; ++w) {
            const float wt = s_ml[w][hh][0] == -INFINITY ? (s_ml[w][hh][1] == 0.f ? 0.f : 1.f) : expf(s_ml[w][hh][0] - M);
            L = fmaf(s_ml[w][hh][1], wt, L);
            acc = fmaf(s_o[((size_t)w * A.g + hh) * kHeadDim + i % kHeadDim], wt, acc);
        }
        const size_t row = (size_t)b * A.hq + (size_t)h * A.g + hh;
        A.O[row * kHeadDim + i % kHeadDim] = L == 0.f ? 0.f : acc / L;
        if (A.lse && i % kHeadDim == 0) A.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
    }
}

}  // namespace

size_t attn4_workspace(const ice_params &) { return 256; }

cudaError_t launch_attn4(const ice_params &p, const void *Q, const void *records, const int32_t *page_len,
                         const int32_t *sel_pages, const int32_t *sel_count, int max_sel, const ice_cache4 *cache,
                         const int32_t *lens, float scale, float *O, float *lse, void *ws, int32_t *err,
                         cudaStream_t s) {
    (void)ws;
    Attn4Args A{};
    A.Q = Q;
    A.pool = static_cast<const unsigned char *>(records);
    A.page_len = page_len, A.sel_pages = sel_pages, A.sel_count = sel_count;
    A.page_cap = p.page_cap, A.max_sel = max_sel;
    if (cache) {
        A.cache = static_cast<const unsigned char *>(cache->records);
        A.table = cache->table, A.n_pages = cache->n_pages, A.max_pages = cache->max_pages;
        A.lens = lens;
    }
    A.g = p.n_q_heads / p.n_kv_heads, A.hq = p.n_q_heads, A.hkv = p.n_kv_heads;
    A.scale = scale;
    A.O = O, A.lse = lse, A.err = err;
    const size_t smem = sizeof(float) * kWarps * A.g * kHeadDim;
    auto kern = p.dtype == ICE_BF16 ? k_attn4<__nv_bfloat16> : k_attn4<float>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(units_of(p)), dim3(kWarps * 32), smem, s, A);
}

}  // namespace ice
