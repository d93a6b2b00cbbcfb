// Queries, keys and values from a layer's projection: the norm per head and
// the position rotation in one pass (ice_qkv_rope), and the same with K and V
// appended to a paged cache in 4 bits (ice_cache4_append).
//
//   norm      y = (x r) w, r = 1 / sqrt(mean(x^2) + eps).  Keys take the sum
//             of squares as an error-free double-float sum (a 4-bit code may
//             hang on its last bit), queries as a plain fp32 sum;
//   rotation  (a, b) <- (a cos - b sin, b cos + a sin), each product rounded
//             once (no contraction).  Keys of an fp32 cache take the products
//             with their rounding errors: their codes hang on the last bit.
//
// Prompts are bound by HBM, each row read and written once: 1 x 36k tokens of
// 32/8 heads 137 us, 6.75 TB/s, the copy rate.  With norms the sums share the
// bound: 1 x 20k tokens of 64/8 heads 140 us, 5.9 TB/s (150 us with error-free
// sums for the queries too).  Single tokens are bound by latency: 3.2 us for 16
// sequences.
//
// 8 lanes hold a row as two 8-element vectors: for pairs (i, i + rotary_dim /
// 2) vectors l and l + rotary_dim / 16, so that both elements of a pair are in
// one lane and nothing is exchanged but the norm's sum.  k_qkv_rope: 8 lanes
// take four heads of one token, whose cos and sin stay in registers; all loads
// are issued before the arithmetic.
//
// k_cache4_append: CTAs of the queries work that way; in the others a warp per
// block of 16 cache slots and KV head quantises up to 16 rows, four at a time,
// into a record in shared memory, and writes the record (all 16 slots new) or
// only the new tokens' bytes of it; with few blocks a warp takes four slots.
// The quantising CTAs are bound by their instructions (alone: 23 us, 3.0 TB/s),
// those of the queries by HBM, so both kinds run side by side: the former lie
// evenly among the first three quarters of the grid, and what is left at the
// end is short.  Appending 4 x 4099 tokens of 32/8 heads: 49.9 us (5.8 TB/s);
// spread over the whole grid 52.9, queries first 54.8, K and V first 53.2.
//
// Other forms, 1 x 16k tokens of 64/8 heads (floors 100 and 106 us): rotation in
// halves 100 us, with norms 117, pairs (2 i, 2 i + 1) 112, 64 of 128 elements
// 113, the former with norms 124; append with its read 112, 135, 129, 133 and
// 148 (the kernels with norms or other rotations spill 76 to 324 bytes).
//
// The launch bounds trade registers for warps: at least 6 CTAs (24 warps) an SM
// in bf16 (the 36k prompt 159 us with 4, the same with 8; the append 56 us with
// 4, 52 with 8), in fp32 3 for the rotation (4 the same, 5 155 us instead of 146
// for 20k tokens) and 4 for the append (20k tokens 129 us; with 3 139, without
// a bound 167).
#include "common.cuh"
#include "internal.h"
#include "quant4.cuh"
#include "tc_common.cuh"

namespace ice {
namespace {

using q4::pair_t;

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;  // rows in flight per CTA
constexpr int kHeads = 4;              // heads per lane group

struct RopeArgs {
    ice_rows q, k, v, qo, ko, vo;
    int hq, hkv, n_new;
    const int32_t *positions, *start, *counts;
    const float *table;
    int n_positions, rotary, interleaved;
    float eps;
    const void *wq, *wk;
    int32_t *err;
};

// The kernels' layouts: bf16 rows rotated as a whole in halves (what the
// models here do), compiled apart from the rest so that its loops are short.
constexpr int kHalves = 0, kAny = 1;

// Which vectors of a row a lane holds, and which of them are rotated.
struct LaneVecs {
    int wa, wb;
    bool ra, rb;
};
template <int kLayout>
__device__ __forceinline__ LaneVecs lane_vecs(const RopeArgs &A, int l) {
    LaneVecs v;
    if (kLayout == kHalves) {
        v.wa = l, v.wb = l + 8, v.ra = v.rb = true;
        return v;
    }
    const int rd = A.table ? A.rotary : 0;
    if (A.interleaved || rd == 0) {
        v.wa = l, v.wb = l + 8;
        v.ra = v.wa * 8 < rd, v.rb = v.wb * 8 < rd;
    } else {
        const int nv = rd / 16;  // vectors of half the rotated elements
        const bool r = l < nv;
        v.wa = r ? l : rd / 8 + 2 * (l - nv);
        v.wb = r ? l + nv : v.wa + 1;
        v.ra = v.rb = r;
    }
    return v;
}

// cos and sin of a lane's 8 pairs.
template <int kLayout>
__device__ __forceinline__ void load_angles(const RopeArgs &A, const LaneVecs &v, int pos, float (&c)[8],
                                            float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    const bool inter = kLayout == kAny && A.interleaved;
    const float *row = A.table + (size_t)pos * (kLayout == kHalves ? kHeadDim : A.rotary);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // pairs 8 wa ..; interleaved: pairs 4 wa .. of vector A, then 4 wb .. of B
        const bool on = inter ? (i < 2 ? v.ra : v.rb) : v.ra;
        const int pair = inter ? (i < 2 ? 4 * v.wa + 2 * i : 4 * v.wb + 2 * (i - 2)) : 8 * v.wa + 2 * i;
        if (on) {
            const float4 f = *reinterpret_cast<const float4 *>(row + 2 * pair);
            c[2 * i] = f.x, s[2 * i] = f.y, c[2 * i + 1] = f.z, s[2 * i + 1] = f.w;
        }
    }
}

// x y + z w, its products and their sum with their rounding errors: within
// 2^-44 of the exact value before the one rounding.
__device__ __forceinline__ float dot2_wide(float x, float y, float z, float w) {
    const float p = __fmul_rn(x, y), q = __fmul_rn(z, w);
    float s, e;
    two_sum(p, q, s, e);
    return s + (e + (fmaf(x, y, -p) + fmaf(z, w, -q)));
}

template <bool kWide>
__device__ __forceinline__ void rotate_pair(float &a, float &b, float c, float s) {
    float x, y;
    if (kWide) {
        x = dot2_wide(a, c, -b, s), y = dot2_wide(b, c, a, s);
    } else {
        x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    }
    a = x, b = y;
}

template <int kLayout, bool kWide>
__device__ __forceinline__ void rotate(const RopeArgs &A, const LaneVecs &v, float (&a)[8], float (&b)[8],
                                       const float (&c)[8], const float (&s)[8]) {
    if (kLayout == kHalves && !kWide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const pair_t x = pk2(a[2 * i], a[2 * i + 1]), y = pk2(b[2 * i], b[2 * i + 1]);
            const pair_t co = pk2(c[2 * i], c[2 * i + 1]), si = pk2(s[2 * i], s[2 * i + 1]);
            // (packed sums of packed products come out fused: the sums stay scalar)
            const float2 p = upk2(mul2(x, co)), q = upk2(mul2(y, si)), u = upk2(mul2(y, co)), w = upk2(mul2(x, si));
            a[2 * i] = __fsub_rn(p.x, q.x), a[2 * i + 1] = __fsub_rn(p.y, q.y);
            b[2 * i] = __fadd_rn(u.x, w.x), b[2 * i + 1] = __fadd_rn(u.y, w.y);
        }
    } else if (A.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (v.ra) rotate_pair<kWide>(a[2 * i], a[2 * i + 1], c[i], s[i]);
            if (v.rb) rotate_pair<kWide>(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
        }
    } else if (v.ra) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate_pair<kWide>(a[e], b[e], c[e], s[e]);
    }
}

// x <- (x r) w over the 8 lanes of a row (every lane of the warp calls it).
// Keys take the error-free sum (their 4-bit codes may hang on its last bit),
// queries a plain fp32 sum.
template <typename T, bool kExact>
__device__ __forceinline__ void norm_row(float (&a)[8], float (&b)[8], const float (&wa)[8], const float (&wb)[8],
                                         float eps) {
    pair_t sum2 = pk2(0.f, 0.f), lo2 = sum2;  // two sums, of the even and the odd elements
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const pair_t f = i < 4 ? pk2(a[2 * (i & 3)], a[2 * (i & 3) + 1]) : pk2(b[2 * (i & 3)], b[2 * (i & 3) + 1]);
        if (kExact) {
            // bf16 squares are exact; those of fp32 values are rounded once, as scalars (a packed product that a packed
            // sum takes comes out fused, and its rounding error, added here, would count twice)
            const float2 x = upk2(f);
            const pair_t t = sizeof(T) == 2 ? mul2(f, f) : pk2(__fmul_rn(x.x, x.x), __fmul_rn(x.y, x.y));
            pair_t er;
            two_sum2(sum2, t, sum2, er);
            lo2 = add2(lo2, er);
            if (sizeof(T) == 4) lo2 = add2(lo2, fma2(f, f, sub2(pk2(0.f, 0.f), t)));
        } else {
            sum2 = fma2(f, f, sum2);
        }
    }
    const float2 hh = upk2(sum2), ll = upk2(lo2);
    float sum, lo = 0.f;
    if (kExact) {
        two_sum(hh.x, hh.y, sum, lo);
        lo += ll.x + ll.y;
    } else {
        sum = hh.x + hh.y;
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, sum, off);
        if (kExact) {
            const float olo = __shfl_xor_sync(0xffffffffu, lo, off);
            float t, er;
            two_sum(sum, other, t, er);
            sum = t;
            lo += olo + er;
        } else {
            sum += other;
        }
    }
    // an overflowed sum is infinite (its error terms are not numbers): r = 0, as in plain fp32
    if (kExact && isfinite(sum)) sum += lo;
    const float r = __frsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / kHeadDim), eps));
    const pair_t r2 = pk2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = upk2(mul2(mul2(pk2(a[2 * i], a[2 * i + 1]), r2), pk2(wa[2 * i], wa[2 * i + 1])));
        const float2 y = upk2(mul2(mul2(pk2(b[2 * i], b[2 * i + 1]), r2), pk2(wb[2 * i], wb[2 * i + 1])));
        a[2 * i] = x.x, a[2 * i + 1] = x.y, b[2 * i] = y.x, b[2 * i + 1] = y.y;
    }
}

// Position of token i of sequence b; -1 when the table does not hold it.
__device__ __forceinline__ int position_of(const RopeArgs &A, int b, int i) {
    if (!A.table) return 0;
    const long long pos = A.positions ? (long long)A.positions[(size_t)b * A.n_new + i]
                                      : (long long)(A.start ? A.start[b] : 0) + i;
    return pos >= 0 && pos < A.n_positions ? (int)pos : -1;
}

__device__ __forceinline__ int count_of(const RopeArgs &A, int b) {
    return A.counts ? min(max(A.counts[b], 0), A.n_new) : A.n_new;
}

// What a CTA's rows are.
constexpr int kQ = 0, kK = 1, kV = 2;

// Item `item` of `items`: kHeads heads of one token of q, k or v.
template <typename T, int kLayout, bool kNorm, int kKind>
__device__ __forceinline__ void dense_chunk(const RopeArgs &A, unsigned item, unsigned items) {
    const int l = threadIdx.x & 7;
    const ice_rows &in = kKind == kQ ? A.q : (kKind == kK ? A.k : A.v);
    const ice_rows &out = kKind == kQ ? A.qo : (kKind == kK ? A.ko : A.vo);
    const int heads = kKind == kQ ? A.hq : A.hkv;
    const unsigned chunks = (heads + kHeads - 1) / kHeads;
    bool live = item < items;  // (every lane stays: the norm shuffles)
    if (!live) item = 0;
    const unsigned tok = item / chunks;
    const int b = tok / A.n_new, i = tok % A.n_new, h0 = (int)(item % chunks) * kHeads;
    live = live && i < count_of(A, b);
    const LaneVecs v = lane_vecs<kLayout>(A, l);
    const T *src = static_cast<const T *>(in.data) + (long long)b * in.batch + (long long)i * in.token;
    T *dst = static_cast<T *>(out.data) + (long long)b * out.batch + (long long)i * out.token;
    q4::Vec8<T> ra[kHeads], rb[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        ra[j].zero();
        rb[j].zero();
        if (live && h0 + j < heads) {
            ra[j].load(src + (h0 + j) * in.head + v.wa * 8);
            rb[j].load(src + (h0 + j) * in.head + v.wb * 8);
        }
    }
    const int pos = live ? position_of(A, b, i) : 0;
    if (pos < 0) {
        set_err(A.err, ICE_ERR_CAPACITY);
        live = false;
    }
    const bool turn = live && kKind != kV && (kLayout == kHalves || A.table);
    float co[8], si[8];
    if (turn) load_angles<kLayout>(A, v, pos, co, si);
    const T *w = static_cast<const T *>(kKind == kQ ? A.wq : A.wk);
    const bool norm = kNorm && kKind != kV && w;
    float wa[8] = {}, wb[8] = {};
    if (norm) {
        load8<T>(w + v.wa * 8, wa);
        load8<T>(w + v.wb * 8, wb);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        float a[8], c[8];
        ra[j].get(a);
        rb[j].get(c);
        if (norm) norm_row<T, kKind == kK>(a, c, wa, wb, A.eps);
        if (turn) rotate<kLayout, false>(A, v, a, c, co, si);
        if (live && h0 + j < heads) {
            store8<T>(dst + (h0 + j) * out.head + v.wa * 8, a);
            store8<T>(dst + (h0 + j) * out.head + v.wb * 8, c);
        }
    }
}

// CTAs [0, q_blocks) take the queries, the next k_blocks the keys, the rest the
// values.
template <typename T, int kLayout, bool kNorm>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 6) k_qkv_rope(
    const __grid_constant__ RopeArgs A, unsigned q_items, unsigned kv_items, int q_blocks, int k_blocks) {
    dep_wait();
    const int block = blockIdx.x;
    const unsigned group = threadIdx.x / 8;
    if (block < q_blocks)
        dense_chunk<T, kLayout, kNorm, kQ>(A, block * kGroups + group, q_items);
    else if (block < q_blocks + k_blocks)
        dense_chunk<T, kLayout, kNorm, kK>(A, (block - q_blocks) * kGroups + group, kv_items);
    else
        dense_chunk<T, kLayout, kNorm, kV>(A, (block - q_blocks - k_blocks) * kGroups + group, kv_items);
}

template <typename T, int kLayout, bool kNorm>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : 6) k_cache4_append(
    const __grid_constant__ RopeArgs A, unsigned q_items, unsigned spread, unsigned kv_blocks, unsigned n_items,
    int blocks, bool split, unsigned char *__restrict__ records, const int32_t *__restrict__ table, int n_pages,
    int max_pages) {
    __shared__ __align__(16) unsigned char s_rec[kThreads / 32][q4::kRecord];
    dep_wait();
    // K and V CTAs before this one
    const unsigned kv = spread ? min(__umulhi(blockIdx.x, spread), kv_blocks) : blockIdx.x;
    if (spread && min(__umulhi(blockIdx.x + 1, spread), kv_blocks) == kv) {  // the queries
        dense_chunk<T, kLayout, kNorm, kQ>(A, (blockIdx.x - kv) * kGroups + threadIdx.x / 8, q_items);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 3, l = lane & 7;
    unsigned item = kv * (kThreads / 32) + warp;
    if (item >= n_items) return;
    const int part = split ? (int)(item & 3u) : 0;  // four of the block's slots, when it is split
    if (split) item >>= 2;
    const int h = (int)(item % A.hkv);
    const int x = (int)(item / A.hkv % blocks);
    const int b = (int)(item / A.hkv / blocks);
    const long long s0 = A.start[b];
    const int cnt = count_of(A, b);
    const long long blk = (s0 >> 4) + x;  // block of 16 cache slots (floor also for a negative start)
    const long long t0 = blk * kPage;
    const long long p0 = t0 + 4 * part, p1 = split ? p0 + 4 : t0 + kPage;
    const long long ta = p0 > s0 ? p0 : s0, tb = p1 < s0 + cnt ? p1 : s0 + cnt;
    if (ta >= tb) return;
    int pg = -1;
    if (blk >= 0 && blk < max_pages) pg = table[(size_t)b * max_pages + blk];
    if (pg < 0 || pg >= n_pages) {
        if (lane == 0) set_err(A.err, ICE_ERR_CAPACITY);
        return;
    }
    unsigned char *rec = s_rec[warp];
    const LaneVecs v = lane_vecs<kLayout>(A, l);
    const T *w = static_cast<const T *>(A.wk);
    float wa[8] = {}, wb[8] = {};
    if (kNorm && w) {
        load8<T>(w + v.wa * 8, wa);
        load8<T>(w + v.wb * 8, wb);
    }
    unsigned done = 0;  // tokens of the block that are written
    const T *kb = static_cast<const T *>(A.k.data) + b * A.k.batch + h * A.k.head;
    const T *vb = static_cast<const T *>(A.v.data) + b * A.v.batch + h * A.v.head;
    struct Rows {
        q4::Vec8<T> ka, kb, va, vb;
    };
    auto load = [&](int it, Rows &x) {  // (lanes without a new token: the nearest one's rows)
        const long long t = t0 + it * 4 + row;
        const long long i = (t < ta ? ta : (t < tb ? t : tb - 1)) - s0;
        const T *ks = kb + i * A.k.token, *vs = vb + i * A.v.token;
        x.ka.load(ks + v.wa * 8);
        x.kb.load(ks + v.wb * 8);
        x.va.load(vs + l * 8);
        x.vb.load(vs + (l + 8) * 8);
    };
    // four rows a turn, the next turn's in flight; rolled, to stay in the instruction cache
    const int last = (int)(tb - 1 - t0) >> 2;
    Rows cur, next;
    load((int)(ta - t0) >> 2, cur);
#pragma unroll 1
    for (int it = (int)(ta - t0) >> 2; it <= last; ++it) {
        const int t = it * 4 + row;
        bool live = t0 + t >= ta && t0 + t < tb;
        const int pos = live ? position_of(A, b, (int)(t0 + t - s0)) : 0;
        if (it < last) load(it + 1, next);
        if (pos < 0) {
            set_err(A.err, ICE_ERR_CAPACITY);
            live = false;
        }
        const unsigned rows = __ballot_sync(0xffffffffu, live && l == 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) done |= (rows >> (8 * r) & 1u) << (it * 4 + r);
        float a[8], c[8];
        cur.ka.get(a);
        cur.kb.get(c);
        if (kNorm && w) norm_row<T, true>(a, c, wa, wb, A.eps);
        if (kLayout == kHalves || A.table) {
            float co[8], si[8];
            load_angles<kLayout>(A, v, max(pos, 0), co, si);
            rotate<kLayout, sizeof(T) == 4>(A, v, a, c, co, si);
        }
        cur.ka.set(a);  // rounded to the storage type
        cur.kb.set(c);
        uint32_t ca, cb;
        uint2 meta;
        q4::quantise_row<T>(cur.ka, cur.kb, v.wa, v.wb, live, ca, cb, meta);
        q4::put_k(rec, t, v.wa, v.wb, ca, cb);
        if (l == 0) *reinterpret_cast<uint2 *>(rec + q4::kKMeta + t * 8) = meta;
        q4::quantise_row<T>(cur.va, cur.vb, l, l + 8, live, ca, cb, meta);
        q4::put_v(rec, t, l, l + 8, ca, cb);
        if (l == 0) *reinterpret_cast<uint2 *>(rec + q4::kVMeta + t * 8) = meta;
        cur = next;
    }
    __syncwarp();
    unsigned char *out = records + ((size_t)pg * A.hkv + h) * q4::kRecord;
    if (done == 0xFFFFu) {
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {  // one bulk store; the buffer has been read before the CTA ends
            tc::bulk_store(out, rec, q4::kRecord);
            tc::bulk_commit();
            tc::bulk_wait_read_all();
        }
        return;
    }
    // only the new tokens: K rows of four 16-byte vectors, the (step, mid) pairs, V in 2-byte pieces
#pragma unroll
    for (int i = lane; i < kPage * 4; i += 32)
        if (done >> (i >> 2) & 1u) reinterpret_cast<uint4 *>(out)[i] = reinterpret_cast<const uint4 *>(rec)[i];
    {
        const int t = lane & 15, off = (lane < 16 ? q4::kKMeta : q4::kVMeta) + t * 8;
        if (done >> t & 1u) *reinterpret_cast<uint2 *>(out + off) = *reinterpret_cast<const uint2 *>(rec + off);
    }
    for (unsigned m = done; m; m &= m - 1) {
        const int off = q4::v_piece(__ffs(m) - 1, lane);
        *reinterpret_cast<uint16_t *>(out + off) = *reinterpret_cast<const uint16_t *>(rec + off);
    }
}

__global__ void k_rope_table(const double *__restrict__ inv_freq, int half, long long n, float2 *__restrict__ table) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    double s, c;
    sincos((double)(i / half) * inv_freq[i % half], &s, &c);
    table[i] = make_float2((float)c, (float)s);
}

RopeArgs rope_args(const ice_params &p, int n_new, const ice_rows *q, const ice_rows *k, const ice_rows *v,
                   const int32_t *positions, const int32_t *start, const int32_t *counts, const ice_rope *rope,
                   const ice_rows *q_out, const ice_rows *k_out, const ice_rows *v_out, int32_t *err) {
    RopeArgs A{};
    if (q) A.q = *q;
    if (k) A.k = *k;
    if (v) A.v = *v;
    if (q_out) A.qo = *q_out;
    if (k_out) A.ko = *k_out;
    if (v_out) A.vo = *v_out;
    A.hq = p.n_q_heads;
    A.hkv = p.n_kv_heads;
    A.n_new = n_new;
    A.positions = positions;
    A.start = start;
    A.counts = counts;
    if (rope) {
        A.table = rope->table;
        A.n_positions = rope->n_positions;
        A.rotary = rope->rotary_dim;
        A.interleaved = rope->interleaved;
        A.eps = rope->eps;
        A.wq = rope->q_norm;
        A.wk = rope->k_norm;
    }
    A.err = err;
    return A;
}

// The instantiation for a call: bf16 in halves without or with norms, bf16 with
// any other rotation, fp32.
template <typename K> K pick(const ice_params &p, const RopeArgs &A, K halves, K halves_norm, K any, K fp32) {
    if (p.dtype != ICE_BF16) return fp32;
    if (!A.table || A.interleaved || A.rotary != kHeadDim) return any;
    return A.wq || A.wk ? halves_norm : halves;
}

}  // namespace

cudaError_t launch_rope_table(const double *inv_freq, int rotary_dim, int n_positions, float *table, cudaStream_t s) {
    const long long n = (long long)n_positions * (rotary_dim / 2);
    k_rope_table<<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(inv_freq, rotary_dim / 2, n,
                                                           reinterpret_cast<float2 *>(table));
    return cudaGetLastError();
}

cudaError_t launch_qkv_rope(const ice_params &p, int n_new, const ice_rows *q, const ice_rows *k, const ice_rows *v,
                            const int32_t *positions, const int32_t *start, const int32_t *counts,
                            const ice_rope *rope, const ice_rows *q_out, const ice_rows *k_out, const ice_rows *v_out,
                            int32_t *err, cudaStream_t s) {
    RopeArgs A = rope_args(p, n_new, q, k, v, positions, start, counts, rope, q_out, k_out, v_out, err);
    const long long toks = (long long)p.batch * n_new;
    const unsigned q_items = (unsigned)(q ? toks * ceil_div(p.n_q_heads, kHeads) : 0);
    const unsigned kv_items = (unsigned)(toks * ceil_div(p.n_kv_heads, kHeads));
    const int q_blocks = ceil_div(q_items, kGroups), k_blocks = k ? ceil_div(kv_items, kGroups) : 0;
    const dim3 grid(q_blocks + k_blocks + (v ? ceil_div(kv_items, kGroups) : 0));
    if (grid.x == 0) return cudaSuccess;
    auto kern = pick(p, A, k_qkv_rope<__nv_bfloat16, kHalves, false>, k_qkv_rope<__nv_bfloat16, kHalves, true>,
                     k_qkv_rope<__nv_bfloat16, kAny, true>, k_qkv_rope<float, kAny, true>);
    return launch_dependent(kern, grid, dim3(kThreads), 0, s, A, q_items, kv_items, q_blocks, k_blocks);
}

cudaError_t launch_cache4_append(const ice_params &p, int n_new, const ice_rows *q, const ice_rows *k,
                                 const ice_rows *v, const int32_t *positions, const int32_t *start,
                                 const int32_t *counts, const ice_rope *rope, const ice_rows *q_out,
                                 const ice_cache4 &cache, int32_t *err, cudaStream_t s) {
    RopeArgs A = rope_args(p, n_new, q, k, v, positions, start, counts, rope, q_out, nullptr, nullptr, err);
    const unsigned q_items = (unsigned)(q ? (long long)p.batch * n_new * ceil_div(p.n_q_heads, kHeads) : 0);
    const unsigned q_blocks = (unsigned)ceil_div(q_items, kGroups);
    const int blocks = cache4_blocks(n_new);
    unsigned items = (unsigned)((long long)p.batch * blocks * p.n_kv_heads);
    // Few blocks leave most of an SM's warps empty while each works on its 16 rows: a warp then takes four of them.  In
    // bf16 1 x 128 tokens of 8 heads take 3.4 us so, 6.2 with whole blocks; 2 x 1200 8.7 and 12.6, 4 x 1200 (16 blocks
    // an SM) 14.7 and 15.0, 8 x 1200 31 and 28.  fp32: 1 x 128 4.0 and 7.7, 4 x 1200 27.6 and 27.1, 8 x 1200 54 and 48.
    const bool split = n_new > 4 && (long long)items <= 16 * device_sms();
    if (split) items *= 4;
    const unsigned kv_blocks = (unsigned)ceil_div(items, kThreads / 32), n = q_blocks + kv_blocks;
    // min(floor(i spread / 2^32), kv_blocks) CTAs of K and V come before CTA i: none before CTA 0, one more after at
    // most every CTA (spread < 2^32), all of them before CTA `over` <= n
    const unsigned over = max(kv_blocks + 1, n / 4 * 3);
    const unsigned spread = q_blocks ? (unsigned)(((unsigned long long)kv_blocks << 32) / over + 1) : 0u;
    const dim3 grid(n);
    unsigned char *r = static_cast<unsigned char *>(cache.records);
    auto kern = pick(p, A, k_cache4_append<__nv_bfloat16, kHalves, false>, k_cache4_append<__nv_bfloat16, kHalves, true>,
                     k_cache4_append<__nv_bfloat16, kAny, true>, k_cache4_append<float, kAny, true>);
    return launch_dependent(kern, grid, dim3(kThreads), 0, s, A, q_items, spread, kv_blocks, items, blocks, split, r,
                            cache.table, cache.n_pages, cache.max_pages);
}

}  // namespace ice
