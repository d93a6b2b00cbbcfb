// Semantic pages to 4-bit records and back, and rows out of a 4-bit cache.
//
// ice_pool4_pack: page pg of a unit -> its record; group extremes, step, mid
// and codes as in ice.h.  ice_pool4_unpack and ice_cache4_read: mid + step
// (code - 7.5), rounded to the storage type.
//
// All three move each page once: a bf16 page is 8192 bytes, its record 2304.
// One warp per page: 8 lanes a row (two 16-byte vectors of a bf16 row each),
// four rows at a time; the record is put together (or taken apart) in shared
// memory, because its V part interleaves two tokens, and moved in 16-byte
// vectors (the finished record by one bulk store).  32 units x 12487 pages (4.2
// GB): pack 710 us, 5.91 TB/s, next to HBM bound by issue (1720 instructions a
// page, the schedulers 76% busy); unpack 602 us, 6.96 TB/s (the copy rate is
// 6.78).  8 units x 2017 pages (170 MB): 34 and 28 us.  fp32, 8 units x 6001
// pages (0.9 GB): 121 and 135 us.  Rows of 4 x 4099 tokens of 8 heads leave a
// cache in 11.3 us, 6.2 TB/s.
#include "common.cuh"
#include "internal.h"
#include "quant4.cuh"
#include "tc_common.cuh"

namespace ice {
namespace {

constexpr int kWarps = 4;
constexpr int kVecs = q4::kRecord / 16;

// A page's rows, the first `len` of them, into a record in shared memory: K's
// in four turns of four rows, then V's.  The next turn's loads are in flight
// while one is quantised; the loop is not unrolled, so that it stays in the
// instruction cache.
template <typename T>
__device__ __forceinline__ void page_to_record(const T *kp, const T *vp, int len, unsigned char *rec) {
    const int lane = threadIdx.x & 31, row = lane >> 3, l = lane & 7;
    q4::Vec8<T> a[2], b[2];
    auto load = [&](int turn, q4::Vec8<T> &x, q4::Vec8<T> &y) {  // (rows behind the last one: the last one)
        const T *src = (turn < 4 ? kp : vp) + min((turn & 3) * 4 + row, len - 1) * kHeadDim + l * 8;
        x.load(src);
        y.load(src + 64);
    };
    load(0, a[0], b[0]);
#pragma unroll 1
    for (int pair = 0; pair < 4; ++pair) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int turn = 2 * pair + i, t = (turn & 3) * 4 + row;
            if (i == 0 || pair < 3) load(turn + 1, a[i ^ 1], b[i ^ 1]);
            uint32_t ca, cb;
            uint2 meta;
            q4::quantise_row<T>(a[i], b[i], l, l + 8, true, ca, cb, meta);
            if (t >= len) ca = cb = meta.x = meta.y = 0u;  // pad slots
            if (pair < 2)
                q4::put_k(rec, t, l, l + 8, ca, cb);
            else
                q4::put_v(rec, t, l, l + 8, ca, cb);
            if (l == 0) *reinterpret_cast<uint2 *>(rec + (pair < 2 ? q4::kKMeta : q4::kVMeta) + t * 8) = meta;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_pool4_pack(const T *__restrict__ pool_k, const T *__restrict__ pool_v,
                                                            const int32_t *__restrict__ n_pages,
                                                            const int32_t *__restrict__ page_len, int page_cap,
                                                            int per_unit, unsigned char *__restrict__ records) {
    __shared__ __align__(16) unsigned char s_rec[kWarps][q4::kRecord];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int u = blockIdx.x / per_unit, pg = (blockIdx.x % per_unit) * kWarps + warp;
    dep_wait();
    if (pg >= min(n_pages[u], page_cap)) return;
    const size_t at = (size_t)u * page_cap + pg;
    const int len = min(max(page_len[at], 0), kPage);
    if (len > 0)
        page_to_record<T>(pool_k + at * kPage * kHeadDim, pool_v + at * kPage * kHeadDim, len, s_rec[warp]);
    else
        for (int i = lane; i < kVecs; i += 32) reinterpret_cast<uint4 *>(s_rec[warp])[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_proxy_async();
    __syncwarp();
    if (lane == 0) {  // one bulk store a record; the buffer has been read before the CTA ends
        tc::bulk_store(records + at * q4::kRecord, s_rec[warp], q4::kRecord);
        tc::bulk_commit();
        tc::bulk_wait_read_all();
    }
}

// Tokens first .. n_indexed - 1 of every unit, one row of 8 lanes each, a CTA a
// unit: up to 16 tokens of 8 units take 3.5 us, 128 take 11, 1024 72 (a whole
// pack of 8 x 16k tokens 29).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_pool4_tokens(
    const T *__restrict__ pool_k, const T *__restrict__ pool_v, const int32_t *__restrict__ n_indexed,
    const int32_t *__restrict__ token_page, const int32_t *__restrict__ token_slot, int page_cap, int n_cap, int first,
    unsigned char *__restrict__ records, int32_t *__restrict__ err) {
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int u = blockIdx.x;
    dep_wait();
    const int n = min(n_indexed[u], n_cap);
    // whole warps stay in the loop: the quantiser shuffles
    for (int base = first + (threadIdx.x >> 5) * 4; base < n; base += kWarps * 4) {
        const int tok = base + (lane >> 3);
        int pg = -1, slot = 0;
        if (tok < n) {
            pg = token_page[(size_t)u * n_cap + tok];
            slot = token_slot[(size_t)u * n_cap + tok];
            if (pg < 0 || pg >= page_cap || slot < 0 || slot >= kPage) {
                set_err(err, ICE_ERR_CAPACITY);
                pg = -1;
            }
        }
        const size_t at = (size_t)u * page_cap + (pg < 0 ? 0 : pg);
        unsigned char *rec = records + at * q4::kRecord;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const T *src = (which ? pool_v : pool_k) + (at * kPage + slot) * kHeadDim;
            q4::Vec8<T> a, b;
            a.zero();
            b.zero();
            if (pg >= 0) {
                a.load(src + l * 8);
                b.load(src + (l + 8) * 8);
            }
            uint32_t ca, cb;
            uint2 meta;
            q4::quantise_row<T>(a, b, l, l + 8, pg >= 0, ca, cb, meta);
            if (pg < 0) continue;
            if (which)
                q4::put_v(rec, slot, l, l + 8, ca, cb);
            else
                q4::put_k(rec, slot, l, l + 8, ca, cb);
            if (l == 0)
                *reinterpret_cast<uint2 *>(rec + (which ? q4::kVMeta : q4::kKMeta) + slot * 8) = meta;
        }
    }
}

// Stores the K (which = 0) or V row of token t of a record in shared memory (zeros without `live`): lane l of the row's
// 8.  A store covers 128 bytes of a row: two 16-byte vectors of bf16 a lane, four of fp32.
template <typename T>
__device__ __forceinline__ void store_row(const unsigned char *rec, int which, int t, int l, bool live, T *dst) {
    const uint2 m = *reinterpret_cast<const uint2 *>(rec + (which ? q4::kVMeta : q4::kKMeta) + t * 8);
    if (sizeof(T) == 2) {
#pragma unroll
        for (int w = l; w < 16; w += 8) {
            float x[8] = {};
            if (live)
                q4::values_of(which ? q4::get_v(rec, t, w) : q4::get_k(rec, t, w), q4::unpack_meta(w < 8 ? m.x : m.y), x);
            store8<T>(dst + w * 8, x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = 8 * i + l;  // elements 4 p .. 4 p + 3
            float x[4] = {};
            if (live) {
                const uint32_t w = which ? *reinterpret_cast<const uint16_t *>(rec + q4::v_piece(t, p))
                                         : q4::get_k(rec, t, p >> 1) >> (16 * (p & 1));
                q4::values_of(w, q4::unpack_meta(i < 2 ? m.x : m.y), x);
            }
            *reinterpret_cast<float4 *>(dst + 4 * p) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_pool4_unpack(const unsigned char *__restrict__ records,
                                                              const int32_t *__restrict__ n_pages,
                                                              const int32_t *__restrict__ page_len, int page_cap,
                                                              int per_unit, T *__restrict__ pool_k,
                                                              T *__restrict__ pool_v) {
    __shared__ __align__(16) unsigned char s_rec[kWarps][q4::kRecord];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 3, l = lane & 7;
    const int u = blockIdx.x / per_unit, pg = (blockIdx.x % per_unit) * kWarps + warp;
    dep_wait();
    if (pg >= min(n_pages[u], page_cap)) return;
    const size_t at = (size_t)u * page_cap + pg;
    const int len = min(max(page_len[at], 0), kPage);
    const uint4 *src = reinterpret_cast<const uint4 *>(records + at * q4::kRecord);
    uint4 *buf = reinterpret_cast<uint4 *>(s_rec[warp]);
    for (int i = lane; i < kVecs; i += 32) buf[i] = src[i];
    __syncwarp();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        T *dst = (which ? pool_v : pool_k) + at * kPage * kHeadDim;
#pragma unroll
        for (int it = 0; it < kPage / 4; ++it) {
            const int t = it * 4 + row;
            store_row<T>(s_rec[warp], which, t, l, t < len, dst + t * kHeadDim);
        }
    }
}

// Tokens start .. start + count - 1 of a sequence, one warp per block of 16
// cache slots and KV head.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_cache4_read(const unsigned char *__restrict__ records,
                                                             const int32_t *__restrict__ table, int n_pages,
                                                             int max_pages, int n_kv_heads, int blocks, int n_new,
                                                             const int32_t *__restrict__ start,
                                                             const int32_t *__restrict__ counts, ice_rows k_out,
                                                             ice_rows v_out, int32_t *__restrict__ err,
                                                             unsigned n_items) {
    __shared__ __align__(16) unsigned char s_rec[kWarps][q4::kRecord];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 3, l = lane & 7;
    const unsigned item = blockIdx.x * kWarps + warp;
    dep_wait();
    if (item >= n_items) return;
    const int h = (int)(item % n_kv_heads);
    const int x = (int)(item / n_kv_heads % blocks);
    const int b = (int)(item / n_kv_heads / blocks);
    const long long s0 = start[b];
    const int cnt = counts ? min(max(counts[b], 0), n_new) : n_new;
    const long long blk = (s0 >> 4) + x;  // block of 16 cache slots (floor also for a negative start)
    const long long t0 = blk * kPage;
    const long long ta = t0 > s0 ? t0 : s0, tb = t0 + kPage < s0 + cnt ? t0 + kPage : s0 + cnt;
    if (ta >= tb) return;
    int pg = -1;
    if (blk >= 0 && blk < max_pages) pg = table[(size_t)b * max_pages + blk];
    if (pg < 0 || pg >= n_pages) {
        if (lane == 0) set_err(err, ICE_ERR_CAPACITY);
        return;
    }
    const uint4 *src = reinterpret_cast<const uint4 *>(records + ((size_t)pg * n_kv_heads + h) * q4::kRecord);
    uint4 *buf = reinterpret_cast<uint4 *>(s_rec[warp]);
    for (int i = lane; i < kVecs; i += 32) buf[i] = src[i];
    __syncwarp();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const ice_rows &o = which ? v_out : k_out;
#pragma unroll
        for (int it = 0; it < kPage / 4; ++it) {
            const int t = it * 4 + row;
            if (t0 + t < ta || t0 + t >= tb) continue;
            store_row<T>(s_rec[warp], which, t, l, true,
                         static_cast<T *>(o.data) + b * o.batch + (t0 + t - s0) * o.token + h * o.head);
        }
    }
}

template <typename T>
cudaError_t pack_t(const ice_params &p, const ice_index &idx, int first, void *records, int32_t *err, cudaStream_t s) {
    const T *k = static_cast<const T *>(idx.pool_k), *v = static_cast<const T *>(idx.pool_v);
    unsigned char *r = static_cast<unsigned char *>(records);
    if (first > 0)
        return launch_dependent(k_pool4_tokens<T>, dim3(units_of(p)), dim3(kWarps * 32), 0, s, k, v, idx.n_indexed,
                                idx.token_page, idx.token_slot, p.page_cap, p.n_cap, first, r, err);
    const int per_unit = ceil_div(p.page_cap, kWarps);
    return launch_dependent(k_pool4_pack<T>, dim3((unsigned)per_unit * units_of(p)), dim3(kWarps * 32), 0, s, k, v,
                            idx.n_pages, idx.page_len, p.page_cap, per_unit, r);
}

template <typename T>
cudaError_t unpack_t(const ice_params &p, const ice_index &idx, const void *records, cudaStream_t s) {
    const int per_unit = ceil_div(p.page_cap, kWarps);
    return launch_dependent(k_pool4_unpack<T>, dim3((unsigned)per_unit * units_of(p)), dim3(kWarps * 32), 0, s,
                            static_cast<const unsigned char *>(records), idx.n_pages, idx.page_len, p.page_cap,
                            per_unit, static_cast<T *>(idx.pool_k), static_cast<T *>(idx.pool_v));
}

template <typename T>
cudaError_t read_t(const ice_params &p, int n_new, const ice_cache4 &c, const int32_t *start, const int32_t *counts,
                   const ice_rows &k_out, const ice_rows &v_out, int32_t *err, cudaStream_t s) {
    const int blocks = cache4_blocks(n_new);
    const unsigned items = (unsigned)((long long)p.batch * blocks * p.n_kv_heads);
    return launch_dependent(k_cache4_read<T>, dim3((unsigned)ceil_div(items, kWarps)), dim3(kWarps * 32), 0, s,
                            static_cast<const unsigned char *>(c.records), c.table, c.n_pages, c.max_pages,
                            p.n_kv_heads, blocks, n_new, start, counts, k_out, v_out, err, items);
}

}  // namespace

cudaError_t launch_pool4_pack(const ice_params &p, const ice_index &idx, int first_token, void *records, int32_t *err,
                              cudaStream_t s) {
    return p.dtype == ICE_BF16 ? pack_t<__nv_bfloat16>(p, idx, first_token, records, err, s)
                               : pack_t<float>(p, idx, first_token, records, err, s);
}

cudaError_t launch_pool4_unpack(const ice_params &p, const ice_index &idx, const void *records, cudaStream_t s) {
    return p.dtype == ICE_BF16 ? unpack_t<__nv_bfloat16>(p, idx, records, s) : unpack_t<float>(p, idx, records, s);
}

cudaError_t launch_cache4_read(const ice_params &p, int n_new, const ice_cache4 &cache, const int32_t *start,
                               const int32_t *counts, const ice_rows &k_out, const ice_rows &v_out, int32_t *err,
                               cudaStream_t s) {
    return p.dtype == ICE_BF16 ? read_t<__nv_bfloat16>(p, n_new, cache, start, counts, k_out, v_out, err, s)
                               : read_t<float>(p, n_new, cache, start, counts, k_out, v_out, err, s);
}

}  // namespace ice
