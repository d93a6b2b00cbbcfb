// Attention of one query token over 4-bit pages: ice_cache4_attn_decode (a
// token-ordered cache) and ice_sparse_attn_decode4 (selected pages of a pool,
// then a cache's tokens, in one softmax).
//   O = sum_j exp(scale q . k_j) v_j / sum_j exp(scale q . k_j),
// papernotes.org "IceCache: Memory-Efficient KV-cache Management for
// Long-Sequence LLMs", 关键设计 1, over the unit's pages only.
//
// A page of 16 tokens of one KV head is one 2304-byte record, read once; at the
// measured copy rate an SM could get one every ~98 clocks.  Long caches are
// bound by that and by instruction issue in about equal parts: the same loop
// over pages without their copies takes about 110 clocks a page and SM (250
// instructions on four schedulers, 62 clocks, and 24 products that block one for
// 8 clocks each, 48), the copies alone take 305 us where the whole takes 357 us
// (16 sequences x 100k tokens, 64/8 heads: 1.84 GB at 5.2 TB/s, 76% of the copy
// rate; 4 heads a group 334 us).  The products' share grows with 9 to 16 heads a
// group (48 a page; 580 us with 16) and with fp32 queries (32 a page, and K's
// codes centred: 420 us, with 4 heads a group 390).  Short ones are bound by a chain
// of latencies (1 sequence x 16k tokens, 32/8 heads: 13.5 us): counts of the
// units 1.5 us, page numbers 1.0, queries 0.8, first page 1.6, the run's other
// pages 2.5, the warps' join 1.3, the ticket 1.0, the runs' join 2.5.
//
// Work: the pages of all units, one after another, are cut into equal runs,
// one per CTA, whatever the units' lengths; a unit counts kOver pages more
// than it has (what starting and ending one costs), so that many short units
// do not gather in few CTAs.  A unit that a run cuts leaves partial results in
// the workspace, joined by its last CTA in run order (so the bits do not
// depend on timing).  Inside a CTA place f of the run goes to warp f % 8; a
// warp looks up its pages 32 at a time, one a lane, well before their copies
// start, so that its loop over pages does little else than attend.
//
// Per page and warp, with tokens as the rows (M = 16) and the g <= 8 query
// heads as the columns (N = 8) of m16n8k16 products, so that a group of 8
// heads fills the tile:
//   S^T = K Q^T: the record keeps a token's codes in the order of the A
//     fragments, so a lane's 16-byte loads are its fragments.  A code c at bit
//     0 (or 4) of a half is the fp16 number c 2^-24 (c 2^-20): one AND per
//     pair turns codes into operands, nothing is converted; the queries carry
//     the factor 16 between the two.  Each group of 64 has its accumulator:
//     S = sum_groups step (q . c) + (mid - 7.5 step) sum q.
//     (bf16 queries: subnormal operands, whose sums lose some bits, see below;
//     O's relative error is 3.5e-7 where fp32 products leave 3e-7, lse's 7e-8
//     and 3e-8: fewer instructions were worth that.  fp32 queries go in as two
//     fp16 parts, 22 bits, and the codes centred: 2.5e-7.)
//   softmax: the running maximum only moves when a score passes it by 2^8 (one
//     vote per page instead of reductions); sums stay in their lanes until the
//     end of the unit.
//   O^T += V^T (step P)^T: V codes as operands the same way (the record pairs
//     two tokens in a word); step P in fp16 hi + lo parts (22 bits), scaled
//     by a power of two of each head that follows the steps and their weights;
//     the 8 x 8 transposes of P by movmatrix.  A product blocks the scheduler for 8 clocks (24 of them
//     are 43% of the 111 clocks above), so with g <= 4 the columns 4 .. 7 hold
//     heads 0 .. 3 again and take the lo parts: one product a tile instead of
//     two.  The codes go in centred and as normal numbers, (code - 7.5) 2^-10:
//     a mean over many values cancels down to the noise of its sums, and the
//     tensor core aligns subnormal operands by their nominal exponent, which
//     costs six of its bits (relative error of O: 1e-5 with plain codes, 1.2e-6
//     with centred subnormals, 4e-7 so).  sum mid P joins at the end of the
//     unit.
#include <cuda_fp16.h>
#include <float.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "quant4.cuh"
#include "tc_common.cuh"

namespace ice {
namespace {

using namespace tc;

// Pages of a warp's ring: one attended, two on their way (16 sequences x 100k tokens 357 us; with two slots 371, short
// sequences 1% less).
constexpr int kSlots = 3;
constexpr int kBatch = 32;         // places looked up at a time
constexpr int kLenShift = 58;      // device addresses are below 2^57
// Places that a unit takes beside its pages: 61 ragged sequences of 1 to 4097 tokens (488 units) take 31 us with 8,
// 23.5 with 24, 22.1 with 28, 22.8 with 34 and 23.9 with 44; 32 ragged sequences of up to 2000 tokens 15.5 with 28 and
// 11.7 with 34; 128 units of 64 to 128 pages 18.9, 18.4, 18.2 and 17.9.
constexpr int kOver = 34;
constexpr int kUnits = 512;        // units whose page counts a CTA keeps at hand
constexpr int kRow = kHeadDim + 4;  // padded row of the warps' outputs (conflict-free 16-byte stores)
constexpr int kMaxRuns = 384;      // CTAs, at most
// A unit of more than kJoinRows rows of partial results (runs times heads) is joined in two levels, groups of kGroup
// runs by their last CTAs and then the groups: one CTA reads 10 rows a warp and latency, a further ticket costs about 2
// us.  One sequence of 16k tokens of 16/1 heads takes 16.1 us so and 24.2 in one level, of 100k tokens 20.2 and 36.6
// (4/1 heads 15.5 and 24.2); the 38 runs of 4 heads of 16k tokens of 32/8 heads 15.8 in two levels and 13.4 in one.
constexpr int kGroup = 16, kJoinRows = 256;
constexpr int kMinRun = 8;         // places of a run, at least: one page per warp (16 are slower: fewer CTAs at work)

struct Attn4Args {
    const void *Q;
    const unsigned char *pool;  // selected pages (NULL: none)
    const int32_t *page_len, *sel_pages, *sel_count;
    int page_cap, max_sel;
    const unsigned char *cache;  // token-ordered pages (NULL: none)
    const int32_t *table, *lens;
    int n_pages, max_pages;
    int g, hq, hkv, units;
    float scale;
    float *O, *lse;
    float *part_o, *part_ml;
    int32_t *ticket, *group_ticket, *err;
};

// Two CTAs of 8 warps an SM, 128 registers a thread: 16 warps hide a page's latencies behind one another.  12 warps of
// 168 registers take 374 us where these took 369, 20 of 96 (which spill) 404.  More than 8 heads a group need two
// accumulator tiles: one CTA of 8 warps (8 sequences x 100k tokens of 16 heads a group 292 us; 10 warps 341, 12 293).
template <int HN> struct Shape {
    static constexpr int kHeads = 8 * HN;
    static constexpr int kCtas = HN == 1 ? 2 : 1;    // per SM
    static constexpr int kWarps = 8;
    static constexpr int kThreads = 32 * kWarps;
};

// A unit of a run: index i from u0, first page at place `first` (from the run's start), n pages.
struct UnitAt {
    int i, first, n;
    int2 cnt;
    int b;  // sequence
    __device__ __forceinline__ int end() const { return first + n; }
};

// What the CTA's threads share to prepare the queries of a unit.
template <int NQ, int HN> struct QueryScratch {
    uint2 f[NQ][HN][8][32];  // fragments by lane
    float2 sum[8 * HN];
    float factor[8 * HN];
};

template <int NQ, int HN> struct Smem {
    static constexpr int kWarps = Shape<HN>::kWarps;
    unsigned char ring[kWarps][kSlots][q4::kRecord];
    float o[kWarps][Shape<HN>::kHeads][kRow];  // reused for the joining weights
    QueryScratch<NQ, HN> q;
    float4 ml[kWarps][Shape<HN>::kHeads];  // maximum, sum, and each group's sum P mid
    float4 scale[kWarps][HN][4];  // a warp's powers of two on step P, both groups of heads 2 c and 2 c + 1
    float4 most[kWarps][HN][4];  // and the largest step P that they were found for
    int2 units[kUnits];  // (selected pages, cache tokens) of the units from unit `base` on
    unsigned long long page[kWarps][2 * kBatch];  // pages looked up: address | length << kLenShift; 0: no page
    UnitAt look[kWarps];  // a warp's place in its lookups
    long long sum[kWarps];
    long long start0;  // places before unit u0
    int u0, last;
    UnitAt unit;
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// D += A B, and D = A B; m16n8k16, fp16 in (subnormals kept), fp32 accumulate.
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// a > l or b > l or c > m or d > m.
__device__ __forceinline__ bool exceeds(float a, float b, float c, float d, float l, float m) {
    int r;
    asm("{\n\t.reg .pred p;\n\t"
        "setp.gt.f32 p, %1, %5;\n\t"
        "setp.gt.or.f32 p, %2, %5, p;\n\t"
        "setp.gt.or.f32 p, %3, %6, p;\n\t"
        "setp.gt.or.f32 p, %4, %6, p;\n\t"
        "selp.s32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d), "f"(l), "f"(m));
    return r != 0;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (code - 7.5) 2^-10 of two codes at bit 0 (c 2^-24 as fp16) or bit 4 (c 2^-20) of the halves: exact.
__device__ __forceinline__ uint32_t centred(uint32_t x, bool high) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(high ? 0x64006400u : 0x74007400u), "r"(0x9F809F80u));
    return d;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The inverse of a power of two 2^e, -126 <= e <= 126.
__device__ __forceinline__ float inverse_of(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }
// Exponent of a positive finite float (-127 for subnormals).
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

// The running maxima in powers of two, from minus the scores (-FLT_MAX: no score yet).
__device__ __forceinline__ float2 max_of(unsigned long long minus, unsigned long long factor) {
    const float2 m = upk2(mul2(minus, factor));
    return make_float2(fmaxf(-m.x, -FLT_MAX), fmaxf(-m.y, -FLT_MAX));
}

// Pages after which a warp's sums leave the tensor core's accumulators, whose sums truncate: the relative error of O at
// 100k tokens is 8e-7 so, 8e-6 without.
constexpr int kFlush = 32;
constexpr float kLazy = 8.f;  // powers of two that a score may pass the running maximum by
constexpr int kTopScale = 119;  // powers of two on step P, at most
// Codes as fp16 operands: c 2^-24 at bit 0 of a half, c 2^-20 at bit 4.
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;

using q4::pair_t;

// A warp's running state over the pages of one unit.  Lane (r, c) = (lane / 4,
// lane % 4); o[hn][t][0..3]: elements of head 8 hn + 2 c + (i & 1), row r of
// tile t (i < 2) or row r + 8; tile t = 2 j + k, row half i / 2: element
// 32 j + 4 r + 2 k + i / 2.
template <int HN> struct State {
    float o[HN][8][4];
    pair_t minus_m[HN];          // minus the running maximum score (before Queries::factor), heads 2 c and 2 c + 1
    pair_t l[HN];                // sum of P over this lane's tokens
    pair_t off[HN][2];           // sum of P mid, groups 0 and 1, this lane's tokens
    uint32_t scales;             // shared address of the powers of two on step P (Smem::scale) of this lane's heads
    pair_t vscale[HN][2];        // and the powers: in registers with more than 8 heads a group (16 x 100k tokens of 16
                                 // heads 568 us, when loaded every page 608; 8 heads 363 us, when loaded every page 359)
    float vlimit[2];             // of each group: the step that they hold up to
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int hn = 0; hn < HN; ++hn) {
#pragma unroll
            for (int t = 0; t < 8; ++t) o[hn][t][0] = o[hn][t][1] = o[hn][t][2] = o[hn][t][3] = 0.f;
            minus_m[hn] = pk2(FLT_MAX, FLT_MAX);
            l[hn] = off[hn][0] = off[hn][1] = pk2(0.f, 0.f);
        }
        vlimit[0] = vlimit[1] = 0.f;
        for (int hn = 0; hn < HN; ++hn) vscale[hn][0] = vscale[hn][1] = pk2(pow2(kTopScale), pow2(kTopScale));
    }
    __device__ __forceinline__ void load_scales() {
#pragma unroll
        for (int hn = 0; hn < HN; ++hn) {
            const uint4 v = lds128(scales + hn * 64);
            vscale[hn][0] = pk2(__uint_as_float(v.x), __uint_as_float(v.y));
            vscale[hn][1] = pk2(__uint_as_float(v.z), __uint_as_float(v.w));
        }
    }
};

// The group's queries as B fragments (columns = heads), in fp16 after a power
// of two of each head (a head beside one that is far larger, or not finite,
// keeps its bits), and what the scores need of them.
template <int NQ, int HN> struct Queries {
    uint32_t f;           // shared address of this lane's fragments (QueryScratch::f)
    float sum[HN][2][2];  // sum q over a group, in the products' scale, for this lane's columns (heads 2 c, 2 c + 1)
    pair_t factor[HN];    // > 0: scale log2(e) over the powers of two of q and of the codes (its sign goes to q)
};

// Codes of K as operands: c 2^-24 (kLow; kHigh times 16, and its queries over 16), or with fp32 queries centred() ones,
// whose products keep the bits that those queries have.
template <int NQ> constexpr int kCodeScale = NQ > 1 ? 10 : 24;

// This thread's 8 elements of the group's queries: head tid / 16 (kTwice: heads 4 .. 7 are heads 0 .. 3 again),
// elements 8 (tid % 16) ...
template <typename T, bool kTwice>
__device__ __forceinline__ q4::Vec8<T> query_part(const T *Qg, int g) {
    q4::Vec8<T> v;
    v.zero();
    const int head = kTwice ? (threadIdx.x >> 4) & 3 : threadIdx.x >> 4;
    if (head < g) v.load(Qg + head * kHeadDim + (threadIdx.x & 15) * 8);
    return v;
}

// The queries from every thread's part: the CTA's threads convert one vector
// each, every warp then reads its fragments (all of the CTA's threads call it).
template <typename T, int NQ, int HN>
__device__ __forceinline__ void prepare_queries(const q4::Vec8<T> &part, float scale, QueryScratch<NQ, HN> &X,
                                                Queries<NQ, HN> &q) {
    const int tid = threadIdx.x, lane = tid & 31, c = lane & 3;
    const float sl = scale * 1.4426950408889634f;
    float x[8];
    part.get(x);
    float big = 0.f, s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[e]));
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    const int e2 = min(max(14 - exponent_of(big), -113), 126);  // the largest element lands in [2^14, 2^15)
    const float up = sl == 0.f ? 0.f : copysignf(pow2(e2), sl);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], up, s);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int head = tid >> 4, vec = tid & 15;
    if (head < 8 * HN) {
        if ((vec & 7) == 0) (vec ? X.sum[head].y : X.sum[head].x) = s * pow2(-kCodeScale<NQ>);
        if (vec == 0) {
            // a head that is not finite, or whose factor would not be (bf16: |scale q| from 2^117 on), is not a number
            const float f = sl == 0.f ? 1.f : fabsf(sl) * pow2(kCodeScale<NQ>) * pow2(-e2);
            // (and never zero: slots without a token have a score of -inf)
            X.factor[head] = big < INFINITY && f < INFINITY ? fmaxf(f, FLT_MIN) : __int_as_float(0x7fc00000);
        }
        // element 8 vec + e is code e of word vec: half e / 4, nibble e % 4; the nibbles at bit 4 weigh 16 times more
        uint32_t f[NQ][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float w = NQ == 1 && (p & 1) ? 0.0625f * up : up;
            const float a = x[p] * w, b = x[p + 4] * w;
            const __half2 hi = __floats2half2_rn(a, b);
            f[0][p] = h2_bits(hi);
            if (NQ > 1) {  // fp32 queries: the remainder
                const float2 back = __half22float2(hi);
                f[NQ - 1][p] = h2_bits(__floats2half2_rn(a - back.x, b - back.y));
            }
        }
        const int i = vec >> 2, to = (head & 7) * 4 + (vec & 3);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            X.f[n][head >> 3][2 * i][to] = make_uint2(f[n][0], f[n][1]);
            X.f[n][head >> 3][2 * i + 1][to] = make_uint2(f[n][2], f[n][3]);
        }
    }
    __syncthreads();
    q.f = su32(&X.f[0][0][0][lane]);
#pragma unroll
    for (int hn = 0; hn < HN; ++hn) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 sum = X.sum[8 * hn + 2 * c + e];
            q.sum[hn][0][e] = sum.x, q.sum[hn][1][e] = sum.y;
        }
        q.factor[hn] = pk2(X.factor[8 * hn + 2 * c], X.factor[8 * hn + 2 * c + 1]);
    }
}

// Folds one page (record at shared address `rec`, its first `len` slots; whatever the others hold).
template <int NQ, int HN, bool kTwice>
__device__ __forceinline__ void attend_page4(const Queries<NQ, HN> &q, uint32_t rec, int len, State<HN> &st,
                                             Smem<NQ, HN> &S) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    // ---- S^T = K Q^T, an accumulator per group
    float s[HN][4];
    {
        const uint4 k0 = lds128(rec + r * 64 + c * 16), k1 = lds128(rec + 512 + r * 64 + c * 16);
        const uint2 m0 = lds64(rec + q4::kKMeta + r * 8), m1 = lds64(rec + q4::kKMeta + 64 + r * 8);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        float acc[HN][2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t x0 = w0[i] >> (8 * k), x1 = w1[i] >> (8 * k);
                uint32_t a[4] = {x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh};
                if (NQ > 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = centred(a[e], e > 1);
#pragma unroll
                for (int hn = 0; hn < HN; ++hn)
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float(&d)[4] = acc[hn][i >> 1];
                        const uint2 f = lds64(q.f + ((n * HN + hn) * 8 + 2 * i + k) * 256);
                        if ((i & 1) | k | n)
                            mma_add(d, a, f.x, f.y);
                        else
                            mma_first(d, a, f.x, f.y);
                    }
            }
        const float2 g00 = q4::unpack_meta(m0.x), g01 = q4::unpack_meta(m0.y);  // token r
        const float2 g10 = q4::unpack_meta(m1.x), g11 = q4::unpack_meta(m1.y);  // token r + 8
        constexpr float kOff = NQ > 1 ? 0.f : -7.5f;
        const float2 b0 = upk2(fma2(pk2(kOff, kOff), pk2(g00.x, g01.x), pk2(g00.y, g01.y)));
        const float2 b1 = upk2(fma2(pk2(kOff, kOff), pk2(g10.x, g11.x), pk2(g10.y, g11.y)));
#pragma unroll
        for (int hn = 0; hn < HN; ++hn)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[hn][e] = fmaf(g00.x, acc[hn][0][e],
                                fmaf(g01.x, acc[hn][1][e], fmaf(b0.x, q.sum[hn][0][e], b0.y * q.sum[hn][1][e])));
                s[hn][2 + e] = fmaf(g10.x, acc[hn][0][2 + e],
                                    fmaf(g11.x, acc[hn][1][2 + e], fmaf(b1.x, q.sum[hn][0][e], b1.y * q.sum[hn][1][e])));
            }
    }
    uint2 n0 = lds64(rec + q4::kVMeta + r * 8), n1 = lds64(rec + q4::kVMeta + 64 + r * 8);
    if (len < kPage) {  // slots behind the last token may hold anything
        if (r >= len) {
            n0 = make_uint2(0u, 0u);
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) s[hn][0] = s[hn][1] = -INFINITY;
        }
        if (r + 8 >= len) {
            n1 = make_uint2(0u, 0u);
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) s[hn][2] = s[hn][3] = -INFINITY;
        }
    }
    const float2 v00 = q4::unpack_meta(n0.x), v01 = q4::unpack_meta(n0.y);  // (step, mid): token r, groups 0, 1
    const float2 v10 = q4::unpack_meta(n1.x), v11 = q4::unpack_meta(n1.y);  // token r + 8
    // ---- scores from the running maxima, in powers of two (differences first: those of large scores are exact, their
    // products with the factor are not)
    pair_t y[HN][2];
    auto from_max = [&]() {
#pragma unroll
        for (int hn = 0; hn < HN; ++hn)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                y[hn][half] = mul2(add2(pk2(s[hn][2 * half], s[hn][2 * half + 1]), st.minus_m[hn]), q.factor[hn]);
    };
    from_max();
    // ---- the running maxima and the scales of step P, only when one has to move
    bool far = false;
#pragma unroll
    for (int hn = 0; hn < HN; ++hn) {
        const float2 y0 = upk2(y[hn][0]), y1 = upk2(y[hn][1]);
        far |= exceeds(y0.x, y0.y, y1.x, y1.y, kLazy, kLazy);
    }
    // Steps beyond the powers' limit ask for a move only if a step P is beyond 2^15: where the weight is with small values
    // (a first token of values a thousandth of the others'), most pages have such steps (16 sequences x 100k tokens: 371
    // us in place of 354, with a move each time 454)
    auto beyond = [&]() {
        bool any = false;
#pragma unroll
        for (int hn = 0; hn < HN; ++hn) {
            const float4 v4 = S.scale[threadIdx.x >> 5][hn][c];
            const float2 y0 = upk2(y[hn][0]), y1 = upk2(y[hn][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float p0 = exp2_fast(e ? y0.y : y0.x), p1 = exp2_fast(e ? y1.y : y1.x);
                any |= fmaxf(p0 * v00.x, p1 * v10.x) * (e ? v4.z : v4.x) > 32768.f;
                any |= fmaxf(p0 * v01.x, p1 * v11.x) * (e ? v4.w : v4.y) > 32768.f;
            }
        }
        return any;
    };
    if (__any_sync(0xffffffffu, far | exceeds(v00.x, v10.x, v01.x, v11.x, st.vlimit[0], st.vlimit[1])) &&
        (__any_sync(0xffffffffu, far) || __any_sync(0xffffffffu, beyond()))) {
        // the page's largest scores, its largest and smallest steps (not negative: ordered as their bits are)
        float mx[HN][2];
#pragma unroll
        for (int hn = 0; hn < HN; ++hn)
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[hn][e] = fmaxf(s[hn][e], s[hn][2 + e]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
            for (int hn = 0; hn < HN; ++hn)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    mx[hn][e] = fmaxf(mx[hn][e], __shfl_xor_sync(0xffffffffu, mx[hn][e], off));
        const bool live0 = r < len, live1 = r + 8 < len;
        auto largest = [](float x, float y) {
            return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(x, y))));
        };
        auto smallest = [&](float x, float y) {
            return __uint_as_float(__reduce_min_sync(0xffffffffu, min(__float_as_uint(live0 ? x : INFINITY),
                                                                      __float_as_uint(live1 ? y : INFINITY))));
        };
        const float top[2] = {largest(v00.x, v10.x), largest(v01.x, v11.x)};
        const float low[2] = {smallest(v00.x, v10.x), smallest(v01.x, v11.x)};
        float4(*scale)[4] = S.scale[threadIdx.x >> 5], (*most)[4] = S.most[threadIdx.x >> 5];
        // The powers of two on step P: those that the page's steps ask for (steps up to [2^5, 2^6) now, up to 2^7 before a
        // power moves again: with P <= 2^8 below fp16's 2^16), but more where they would put the largest step P that was
        // seen at such a move below 2^-1, 2^24 times fp16's last place (a value row of little weight may be far larger
        // than those that matter).
        auto power_for = [](float step) { return min(5 - exponent_of(step), kTopScale); };  // >= -122
        auto holds_to = [](int e) { return pow2(min(7 - e, 127)); };
        if (st.vlimit[0] == 0.f && low[0] >= 0.125f * top[0] && low[1] >= 0.125f * top[1]) {
            // the first page, of steps that differ little: every head gives one of them a weight of 1 (one sequence of
            // 16k tokens 13.2 us so, 13.8 by the way below)
            const int e0 = power_for(top[0]), e1 = power_for(top[1]);
            const float to0 = pow2(e0), to1 = pow2(e1);
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) {
                const float2 was = upk2(st.minus_m[hn]);
                st.minus_m[hn] = pk2(fminf(was.x, -mx[hn][0]), fminf(was.y, -mx[hn][1]));
                if (r == 0) {
                    scale[hn][c] = make_float4(to0, to1, to0, to1);
                    most[hn][c] = make_float4(low[0], low[1], low[0], low[1]);
                }
            }
            st.vlimit[0] = holds_to(e0), st.vlimit[1] = holds_to(e1);
            from_max();
        } else {
            float al[HN][2];  // factors on the sums
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) {
                const float2 was = upk2(st.minus_m[hn]), factor = upk2(q.factor[hn]);
                const float now[2] = {fminf(was.x, -mx[hn][0]), fminf(was.y, -mx[hn][1])};
                al[hn][0] = exp2_fast((now[0] - was.x) * factor.x), al[hn][1] = exp2_fast((now[1] - was.y) * factor.y);
                st.minus_m[hn] = pk2(now[0], now[1]);
                st.l[hn] = mul2(st.l[hn], pk2(al[hn][0], al[hn][1]));
#pragma unroll
                for (int e = 0; e < 2; ++e) st.off[hn][e] = mul2(st.off[hn][e], pk2(al[hn][e], al[hn][e]));
            }
            from_max();
            uint32_t ps[HN][2];  // exponents of the page's largest step P, both groups
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) {
                const float2 y0 = upk2(y[hn][0]), y1 = upk2(y[hn][1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p0 = exp2_fast(e ? y0.y : y0.x), p1 = exp2_fast(e ? y1.y : y1.x);
                    ps[hn][e] = __float_as_uint(fmaxf(p0 * v00.x, p1 * v10.x)) >> 23 |
                                (__float_as_uint(fmaxf(p0 * v01.x, p1 * v11.x)) >> 23) << 16;
                }
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                for (int hn = 0; hn < HN; ++hn)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        ps[hn][e] = __vmaxu2(ps[hn][e], __shfl_xor_sync(0xffffffffu, ps[hn][e], off));
            int high[2] = {-126, -126};
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) {
                float4 v4 = scale[hn][c], m4 = most[hn][c];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        float &vs = e ? (gr ? v4.w : v4.z) : (gr ? v4.y : v4.x);
                        float &m = e ? (gr ? m4.w : m4.z) : (gr ? m4.y : m4.x);
                        m = fmaxf(m * al[hn][e], __uint_as_float((gr ? ps[hn][e] >> 16 : ps[hn][e] & 0xFFFFu) << 23));
                        const int had = exponent_of(vs);
                        int to = top[gr] > holds_to(had) ? power_for(top[gr]) : had;
                        if (m > 0.f) to = min(max(to, -1 - exponent_of(m)), kTopScale);
                        high[gr] = max(high[gr], to);
                        vs = pow2(to);
                        // (sums that have lost all weight go: their power may rise without end)
                        const float f = al[hn][e] == 0.f ? 0.f : al[hn][e] * pow2(min(max(to - had, -126), 127));
#pragma unroll
                        for (int t = 4 * gr; t < 4 * gr + 4; ++t) st.o[hn][t][e] *= f, st.o[hn][t][2 + e] *= f;
                    }
                __syncwarp();
                if (r == 0) scale[hn][c] = v4, most[hn][c] = m4;
            }
            st.vlimit[0] = holds_to(high[0]), st.vlimit[1] = holds_to(high[1]);
        }
        __syncwarp();
        if (HN > 1) st.load_scales();
    }
    if (HN == 1) st.load_scales();
    // ---- P, and step P of both groups in hi + lo parts, transposed to B fragments
    uint32_t bh[HN][2][2], bl[HN][2][2];  // [group][token half]
    const pair_t f[2] = {pk2(v00.x, v01.x), pk2(v10.x, v11.x)};
    const pair_t b[2] = {pk2(v00.y, v01.y), pk2(v10.y, v11.y)};
#pragma unroll
    for (int hn = 0; hn < HN; ++hn)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float2 z = upk2(y[hn][half]);
            const float p[2] = {exp2_fast(z.x), exp2_fast(z.y)};
            st.l[hn] = add2(st.l[hn], pk2(p[0], p[1]));
            pair_t x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const pair_t pp = pk2(p[e], p[e]);
                st.off[hn][e] = fma2(pp, b[half], st.off[hn][e]);
                x[e] = mul2(mul2(pp, f[half]), st.vscale[hn][e]);
            }
            const float2 x0 = upk2(x[0]), x1 = upk2(x[1]);
            const __half2 h0 = __floats2half2_rn(x0.x, x1.x), h1 = __floats2half2_rn(x0.y, x1.y);
            const float2 w0 = __half22float2(h0), w1 = __half22float2(h1);
            const float2 d0 = upk2(sub2(x[0], pk2(w0.x, w1.x))), d1 = upk2(sub2(x[1], pk2(w0.y, w1.y)));
            const uint32_t l0 = h2_bits(__floats2half2_rn(d0.x, d1.x)), l1 = h2_bits(__floats2half2_rn(d0.y, d1.y));
            if (kTwice) {  // columns 0 .. 3: the hi parts, columns 4 .. 7, of the same heads: the lo parts
                bh[hn][0][half] = transpose8(c < 2 ? h2_bits(h0) : l0);
                bh[hn][1][half] = transpose8(c < 2 ? h2_bits(h1) : l1);
            } else {
                bh[hn][0][half] = transpose8(h2_bits(h0));
                bh[hn][1][half] = transpose8(h2_bits(h1));
                bl[hn][0][half] = transpose8(l0);
                bl[hn][1][half] = transpose8(l1);
            }
        }
    // ---- O^T += V^T (step P)^T
    {
        const uint4 x0 = lds128(rec + q4::kV + c * 128 + r * 16), x1 = lds128(rec + q4::kV + 512 + c * 128 + r * 16);
        const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t y0 = w0[j] >> (8 * k), y1 = w1[j] >> (8 * k);
                const uint32_t a[4] = {centred(y0 & kLow, false), centred(y0 & kHigh, true),
                                       centred(y1 & kLow, false), centred(y1 & kHigh, true)};
#pragma unroll
                for (int hn = 0; hn < HN; ++hn) {
                    float(&o)[4] = st.o[hn][2 * j + k];
                    mma_add(o, a, bh[hn][j >> 1][0], bh[hn][j >> 1][1]);
                    if (!kTwice) mma_add(o, a, bl[hn][j >> 1][0], bl[hn][j >> 1][1]);
                }
            }
    }
}

// (selected pages, cache tokens) of a unit, within the arrays' bounds.
__device__ __forceinline__ int2 unit_counts(const Attn4Args &A, int u) {
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
// Places of a unit of n pages: kOver, then the pages; none without pages.
__device__ __forceinline__ int places_of(int n) { return n > 0 ? n + kOver : 0; }

// One record (address behind the length bits) into shared memory, by the
// lanes of a warp in 16-byte pieces, as one group; nothing for place entry 0.
// (One bulk copy per page with an mbarrier costs 52 instructions a page more
// in waits and phases: 379 us instead of 369.)
__device__ __forceinline__ void copy_record(uint32_t dst, unsigned long long entry) {
    const int lane = threadIdx.x & 31;
    if (entry != 0) {
        const unsigned char *src = reinterpret_cast<const unsigned char *>(entry & ((1ull << kLenShift) - 1)) + lane * 16;
        dst += lane * 16;
#pragma unroll
        for (int i = 0; i < q4::kRecord / 512; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * i), "l"(src + 512 * i) : "memory");
        if (lane < q4::kRecord % 512 / 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + q4::kRecord / 512 * 512),
                         "l"(src + q4::kRecord / 512 * 512)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Row of O and lse from the sums over all pages (this lane's 4 elements).
__device__ __forceinline__ void put_row(const Attn4Args &A, size_t row, float4 acc, float M, float L) {
    const int lane = threadIdx.x & 31;
    const float inv = L > 0.f ? 1.f / L : L;  // no token: 0; NaN stays
    if (L == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4 *>(A.O + row * kHeadDim + 4 * lane) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (A.lse && lane == 0) A.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Whether this CTA is the last of n to come here (all of its threads call; what the others wrote can then be read).
__device__ __forceinline__ bool last_of(int32_t *ticket, int n, int *last) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();  // (the whole CTA's stores: they come before the barrier)
        *last = atomicAdd(ticket, 1) == n - 1;
    }
    __syncthreads();
    if (!*last) return false;
    __threadfence();
    return true;
}

// Sums of n parts (rows of [.., 128] and (maximum, sum) pairs): the first one's rows at `first`, the others' at k *
// stride.  put(head, acc, M, L) is called by one warp a head, a lane's 4 elements each.
template <int kWarps, typename Put>
__device__ __forceinline__ void join_parts(float *scratch, const float *po, const float2 *ml, int first, int stride,
                                           int n, int g, Put put) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a head's parts go to as many warps as there are for it, whose sums meet in shared memory
    const int split = g >= kWarps ? 1 : kWarps / g;
    float2 *wt = reinterpret_cast<float2 *>(scratch) + warp * kMaxRuns;  // of this warp's head
    float *sums = scratch + 2 * kWarps * kMaxRuns;
    float M, L;
    float4 acc;
    for (int hh = warp / split; hh < g; hh += split == 1 ? kWarps : g) {
        // the first rows are on their way while the weights are found
        constexpr int kAhead = 10;
        const int k0 = warp % split;
        const float4 *row = reinterpret_cast<const float4 *>(po + (size_t)hh * kHeadDim) + lane;
        auto row_of = [&](int k) {
            return k < n ? __ldcg(row + (size_t)(k * stride + (k ? 0 : first)) * (kHeadDim / 4))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float4 y[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) y[i] = row_of(k0 + i * split);
        M = -FLT_MAX, L = 0.f;
        __syncwarp();  // the weights of the head before have been read
        for (int k = lane; k < n; k += 32) {
            const float2 x = __ldcg(ml + k * stride + (k ? 0 : first) + hh);
            M = fmaxf(M, x.x);
            wt[k] = x;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        for (int k = lane; k < n; k += 32) {
            const float2 x = wt[k];
            const float w = x.y == 0.f ? 0.f : (x.y == x.y ? exp2_fast(x.x - M) : x.y);
            L = fmaf(x.y, w, L);
            wt[k].x = w;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
        __syncwarp();
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = k0; k < n; k += kAhead * split) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float w = k + i * split < n ? wt[k + i * split].x : 0.f;
                acc.x = fmaf(y[i].x, w, acc.x), acc.y = fmaf(y[i].y, w, acc.y);
                acc.z = fmaf(y[i].z, w, acc.z), acc.w = fmaf(y[i].w, w, acc.w);
            }
            if (k + kAhead * split < n)
#pragma unroll
                for (int i = 0; i < kAhead; ++i) y[i] = row_of(k + (kAhead + i) * split);
        }
        if (split == 1)
            put(hh, acc, M, L);
        else
            *reinterpret_cast<float4 *>(sums + warp * kHeadDim + 4 * lane) = acc;
    }
    if (split > 1) {  // (at most one head a warp: g <= kWarps / split)
        __syncthreads();
        if (warp % split == 0 && warp / split < g) {
            for (int w = 1; w < split; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(sums + (warp + w) * kHeadDim + 4 * lane);
                acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
            }
            put(warp / split, acc, M, L);
        }
    }
}

// A unit of many runs (the first one's part at 2 ca, or behind it with `inside`): the last CTA of each group of kGroup
// runs joins the group's parts in the place of its first one.  True in those CTAs.  (Not inlined: the loop over pages
// keeps its registers.)
template <int kWarps>
__device__ __noinline__ bool join_group(float *part_o, float *part_ml, int32_t *group_ticket, float *scratch, int *last,
                                        int g, int ca, int runs, bool inside) {
    const int group = ((int)blockIdx.x - ca) / kGroup, from = ca + group * kGroup;
    const bool second = inside && group == 0;
    int32_t *ticket = group_ticket + 2 * from + (second ? 1 : 0);
    const int n = min(kGroup, runs - group * kGroup), first = second ? g : 0;
    if (!last_of(ticket, n, last)) return false;
    float *po = part_o + (size_t)from * 2 * g * kHeadDim;
    float2 *ml = reinterpret_cast<float2 *>(part_ml) + (size_t)from * 2 * g;
    join_parts<kWarps>(scratch, po, ml, first, 2 * g, n, g, [&](int hh, float4 acc, float M, float L) {
        const int lane = threadIdx.x & 31;
        *reinterpret_cast<float4 *>(po + (size_t)(first + hh) * kHeadDim + 4 * lane) = acc;
        if (lane == 0) ml[first + hh] = make_float2(M, L);
    });
    if (threadIdx.x == 0) *ticket = 0;
    return true;
}

template <typename T, int NQ, int HN, bool kTwice>
__global__ void __launch_bounds__(Shape<HN>::kThreads, Shape<HN>::kCtas)
    k_attn4(const __grid_constant__ Attn4Args A) {
    constexpr int kWarps = Shape<HN>::kWarps, kThreads = Shape<HN>::kThreads;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem<NQ, HN> &S = *reinterpret_cast<Smem<NQ, HN> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = A.g;
    dep_wait();

    // ---- the CTA's run of places: a prefix sum over the units
    const bool all = A.units <= kUnits;  // every unit's counts stay at hand
    const int per = (A.units + kThreads - 1) / kThreads;
    const int ua = min(tid * per, A.units), ub = min(ua + per, A.units);
    long long mine = 0;
    for (int u = ua; u < ub; ++u) {
        const int2 cnt = unit_counts(A, u);
        if (all) S.units[u] = cnt;
        const int n = pages_of(cnt);
        mine += places_of(n);
        if (n == 0 && u % (int)gridDim.x == (int)blockIdx.x) {  // no page: nobody else writes these rows
            const size_t row = (size_t)(u / A.hkv) * A.hq + (size_t)(u % A.hkv) * g;
            float4 *o = reinterpret_cast<float4 *>(A.O + row * kHeadDim);
            for (int i = 0; i < g * kHeadDim / 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (A.lse)
                for (int i = 0; i < g; ++i) A.lse[row + i] = -INFINITY;
        }
    }
    long long before = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += y;
    }
    if (lane == 31) S.sum[warp] = before;
    __syncthreads();
    long long total = 0;
    before -= mine;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += S.sum[w];
        total += S.sum[w];
    }
    int share = (int)(total < (1ll << 31) ? ((unsigned)total + gridDim.x - 1) / gridDim.x
                                          : (total + gridDim.x - 1) / gridDim.x);
    if (share < kMinRun) share = kMinRun;
    const long long f0 = (long long)blockIdx.x * share;
    const int run = (int)min((long long)share, total - f0);
    if (run <= 0) return;  // the whole CTA
    if (f0 >= before && f0 < before + mine) {
        long long at = before;
        for (int u = ua; u < ub; ++u) {
            const int n = places_of(pages_of(all ? S.units[u] : unit_counts(A, u)));
            if (f0 < at + n) {
                S.u0 = u;
                S.start0 = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    const int u0 = S.u0, base = all ? 0 : u0;
    if (!all) {
        for (int i = tid; i < kUnits && u0 + i < A.units; i += kThreads) S.units[i] = unit_counts(A, u0 + i);
        __syncthreads();
    }
    auto unit_at = [&](int i, int place) {  // unit u0 + i, whose places start at `place`
        UnitAt x;
        x.i = i;
        x.cnt = u0 - base + i < kUnits ? S.units[u0 - base + i] : unit_counts(A, u0 + i);
        x.n = pages_of(x.cnt);
        x.b = (u0 + i) / A.hkv;
        x.first = place + (x.n > 0 ? kOver : 0);
        return x;
    };
    UnitAt unit = unit_at(0, (int)(S.start0 - f0));
    auto queries_of = [&](const UnitAt &x) {
        const int u = u0 + x.i;
        const size_t row = (size_t)x.b * A.hq + (size_t)(u - x.b * A.hkv) * g;
        return query_part<T, kTwice>(static_cast<const T *>(A.Q) + row * kHeadDim, g);
    };
    q4::Vec8<T> qpart = queries_of(unit);  // in flight during the lookups

    // ---- the warp's pages: places n = 0 .. of the warp are places warp + 8 n of the run
    const int places = run > warp ? (run - warp + kWarps - 1) / kWarps : 0;
    unsigned long long *pages = S.page[warp];
    if (lane == 0) S.look[warp] = unit;
    const uint32_t ring = su32(S.ring[warp][0]);
    auto slot_of = [&](int n) { return ring + (n % kSlots) * q4::kRecord; };
    auto issue = [&](int n, uint32_t to) {  // the copy of place n: one group a place, also where there is no page
        copy_record(to, pages[n & (2 * kBatch - 1)]);
    };
    int looked = 0, issued = 0;  // places looked up, and those whose copy was started
    auto look_further = [&]() {
        __syncwarp();
        UnitAt look = S.look[warp];
        const int n = looked + lane, f = warp + kWarps * n;
        const unsigned char *src = nullptr;
        int len = 0;
        if (n < places) {
            while (f >= look.end()) look = unit_at(look.i + 1, look.end());
            if (f >= look.first) {
                const int x = f - look.first, u = u0 + look.i;
                // a page that does not exist is copied from the first one and attended with length 0
                if (x < look.cnt.x) {
                    src = A.pool;
                    const int id = A.sel_pages[(size_t)u * A.max_sel + x];
                    if (id >= 0 && id < A.page_cap) {
                        const size_t at = (size_t)u * A.page_cap + id;
                        src += at * q4::kRecord;
                        len = A.page_len[at];
                    } else {
                        set_err(A.err, ICE_ERR_CAPACITY);
                    }
                } else {
                    src = A.cache;
                    const int b = look.b, blk = x - look.cnt.x;
                    const int id = A.table[(size_t)b * A.max_pages + blk];
                    if (id >= 0 && id < A.n_pages) {
                        src += ((size_t)id * A.hkv + (u - b * A.hkv)) * q4::kRecord;
                        len = look.cnt.y - blk * kPage;
                    } else {
                        set_err(A.err, ICE_ERR_CAPACITY);
                    }
                }
            }
        }
        unsigned long long *entry = &pages[n & (2 * kBatch - 1)];
        if (looked == 0) {  // the first copies start while the lengths are on their way
            *entry = reinterpret_cast<unsigned long long>(src);
            __syncwarp();
            for (; issued < kSlots - 1; ++issued) issue(issued, slot_of(issued));
            __syncwarp();
        }
        *entry = reinterpret_cast<unsigned long long>(src) | (unsigned long long)min(max(len, 0), kPage) << kLenShift;
        __syncwarp();
        if (lane == 31) S.look[warp] = look;
        looked += kBatch;
        __syncwarp();
    };
    look_further();

    const int r = lane >> 2, c = lane & 3;
    State<HN> st;
    Queries<NQ, HN> q;
    for (bool first = true;; first = false) {
        // the next unit with pages in the run
        while (unit.n == 0 || unit.end() <= 0) unit = unit_at(unit.i + 1, unit.end()), first = false;
        if (unit.first >= run) break;
        if (!first) qpart = queries_of(unit);
        if (tid == 0) S.unit = unit;  // (kept there while the pages take the registers)
        const int pa = max(unit.first, 0), pb = min(unit.end(), run);
        st.init();
        st.scales = su32(&S.scale[warp][0][c]);
        if (lane < 4 * HN) {
            S.most[warp][lane >> 2][lane & 3] = make_float4(0.f, 0.f, 0.f, 0.f);
            S.scale[warp][lane >> 2][lane & 3] =
                make_float4(pow2(kTopScale), pow2(kTopScale), pow2(kTopScale), pow2(kTopScale));
        }
        int n = pa > warp ? (pa - warp + kWarps - 1) / kWarps : 0;
        const int n_end = pb > warp ? (pb - warp + kWarps - 1) / kWarps : 0;
        const bool any = n < n_end;
        if (any)
            for (; issued < n + kSlots - 1; ++issued) {  // (after places without a page)
                if (issued >= looked) look_further();
                issue(issued, slot_of(issued));
            }
        prepare_queries<T, NQ, HN>(qpart, A.scale, S.q, q);
        uint32_t freed = slot_of(n + kSlots - 1), slot = slot_of(n);  // of places n - 1 and n
        for (bool flushed = false; n < n_end; flushed = true) {
            const int until = min(n_end, n + kFlush);
            while (n < until) {
                while (looked - n <= kBatch / 2) look_further();
                const int stop = min(until, looked - (kSlots - 1));
                for (; n < stop; ++n) {
                    // place n has arrived, and every lane is done with n - 1
                    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
                    __syncwarp();
                    issue(n + kSlots - 1, freed);
                    attend_page4<NQ, HN, kTwice>(q, slot, (int)(pages[n & (2 * kBatch - 1)] >> kLenShift), st, S);
                    freed = slot;
                    slot = slot == slot_of(kSlots - 1) ? ring : slot + q4::kRecord;
                }
            }
            issued = n + kSlots - 1;
            __syncwarp();
            // ---- the warp's sums of V to shared memory, in the scale of the running maximum (and times 2^-10, as the codes
            // went in: with that factor too a power of two for the largest steps would overflow)
#pragma unroll
            for (int hn = 0; hn < HN; ++hn) {
                const float2 m2 = max_of(st.minus_m[hn], q.factor[hn]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = 8 * hn + 2 * c + e;
                    const float m = e ? m2.y : m2.x;
                    const float2 vs = *(reinterpret_cast<const float2 *>(&S.scale[warp][hn][c]) + e);
                    const float before = flushed ? exp2_fast(S.ml[warp][head].x - m) : 0.f;
                    __syncwarp();
                    if (r == 0) S.ml[warp][head].x = m;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float(&o0)[4] = st.o[hn][2 * j], (&o1)[4] = st.o[hn][2 * j + 1];
                        const float f = inverse_of(j < 2 ? vs.x : vs.y);
                        float4 *at = reinterpret_cast<float4 *>(&S.o[warp][head][32 * j + 4 * r]);
                        float4 x = make_float4(o0[e] * f, o0[2 + e] * f, o1[e] * f, o1[2 + e] * f);
                        if (flushed) {
                            const float4 y = *at;
                            x.x = fmaf(y.x, before, x.x), x.y = fmaf(y.y, before, x.y);
                            x.z = fmaf(y.z, before, x.z), x.w = fmaf(y.w, before, x.w);
                        }
                        *at = x;
                        o0[e] = o0[2 + e] = o1[e] = o1[2 + e] = 0.f;
                    }
                }
            }
        }
        // ---- and its softmax sums
#pragma unroll
        for (int hn = 0; hn < HN; ++hn) {
            const float2 m2 = max_of(st.minus_m[hn], q.factor[hn]);
            pair_t l2 = st.l[hn], off2[2] = {st.off[hn][0], st.off[hn][1]};
            auto other = [](pair_t x, int by) {
                const float2 y = upk2(x);
                return pk2(__shfl_xor_sync(0xffffffffu, y.x, by), __shfl_xor_sync(0xffffffffu, y.y, by));
            };
            if (any) {
#pragma unroll
                for (int by = 4; by < 32; by <<= 1) {
                    l2 = add2(l2, other(l2, by));
                    off2[0] = add2(off2[0], other(off2[0], by));
                    off2[1] = add2(off2[1], other(off2[1], by));
                }
            }
            if (r == 0) {
                const float2 l = upk2(l2), x = upk2(off2[0]), y = upk2(off2[1]);
                S.ml[warp][8 * hn + 2 * c] = make_float4(m2.x, l.x, x.x, x.y);
                S.ml[warp][8 * hn + 2 * c + 1] = make_float4(m2.y, l.y, y.x, y.y);
            }
        }
        __syncthreads();
        // ---- joined: 32 threads a head, 4 elements each
        unit = S.unit;
        const int u = u0 + unit.i, b = unit.b;
        const size_t row0 = (size_t)b * A.hq + (size_t)(u - b * A.hkv) * g;
        const bool whole = unit.first >= 0 && unit.end() <= run;
        const size_t part = ((size_t)blockIdx.x * 2 + (unit.first > 0 ? 1 : 0)) * g;
        for (int hh = warp; hh < g; hh += kWarps) {
            float M = -FLT_MAX, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, S.ml[w][hh].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 ml = S.ml[w][hh];
                if (ml.y == 0.f) continue;  // no page
                const float wt = ml.y == ml.y ? exp2_fast(ml.x - M) : ml.y;  // a sum that is not a number spreads
                float4 x = *reinterpret_cast<const float4 *>(&S.o[w][hh][4 * lane]);
                if (kTwice) {
                    const float4 y = *reinterpret_cast<const float4 *>(&S.o[w][hh + 4][4 * lane]);
                    x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                }
                const float off = lane < 16 ? ml.z : ml.w;
                L = fmaf(ml.y, wt, L);
                acc.x = fmaf(fmaf(x.x, 1024.f, off), wt, acc.x), acc.y = fmaf(fmaf(x.y, 1024.f, off), wt, acc.y);
                acc.z = fmaf(fmaf(x.z, 1024.f, off), wt, acc.z), acc.w = fmaf(fmaf(x.w, 1024.f, off), wt, acc.w);
            }
            if (whole) {
                put_row(A, row0 + hh, acc, M, L);
            } else {
                *reinterpret_cast<float4 *>(A.part_o + (part + hh) * kHeadDim + 4 * lane) = acc;
                if (lane == 0) *reinterpret_cast<float2 *>(A.part_ml + (part + hh) * 2) = make_float2(M, L);
            }
        }
        if (!whole) {
            // the unit's runs: CTAs ca .. cb; a run's part is its second one when the unit starts inside the run
            const long long us = f0 + unit.first;
            const int ca = (int)(us / share), cb = (int)((us + unit.n - 1) / share);
            const bool inside = us > (long long)ca * share;
            int runs = cb - ca + 1, stride = 2 * g;
            bool go = true;
            if (runs > kGroup && runs * g > kJoinRows) {
                go = join_group<kWarps>(A.part_o, A.part_ml, A.group_ticket, &S.o[0][0][0], &S.last, g, ca, runs,
                                        inside);
                runs = (runs + kGroup - 1) / kGroup, stride *= kGroup;
            }
            if (go && last_of(A.ticket + u, runs, &S.last)) {
                join_parts<kWarps>(&S.o[0][0][0], A.part_o + (size_t)ca * 2 * g * kHeadDim,
                                   reinterpret_cast<const float2 *>(A.part_ml) + (size_t)ca * 2 * g, inside ? g : 0,
                                   stride, runs, g,
                                   [&](int hh, float4 acc, float M, float L) { put_row(A, row0 + hh, acc, M, L); });
                if (tid == 0) A.ticket[u] = 0;
            }
        }
        if (unit.end() >= run) break;
        __syncthreads();  // the results have been read
        unit = unit_at(unit.i + 1, unit.end());
    }
}

int max_ctas(int sms) { return 2 * sms < kMaxRuns ? 2 * sms : kMaxRuns; }

// The partial results lie before the tickets, at sizes that no shape changes:
// calls of different shapes can share a workspace (one after the other) without
// writing over each other's tickets.
struct Attn4Ws {
    float *part_ml;   // [2 runs, g, 2]
    float *part_o;    // [2 runs, g, 128]
    int32_t *group_ticket, *ticket;  // [2 runs], [units]: zero between calls
    size_t bytes;
};
Attn4Ws ws_layout(const ice_params &p, int sms, void *base) {
    Attn4Ws w{};
    char *b = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *r = b ? b + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return r;
    };
    const size_t parts = 2 * (size_t)max_ctas(sms) * 16;  // (g <= 16)
    w.part_ml = reinterpret_cast<float *>(take(sizeof(float) * parts * 2));
    w.part_o = reinterpret_cast<float *>(take(sizeof(float) * parts * kHeadDim));
    w.group_ticket = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * 2 * max_ctas(sms)));
    w.ticket = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * units_of(p)));
    w.bytes = off;
    return w;
}

static_assert(2 * kMaxRuns + kHeadDim <= 8 * kRow, "the joining weights and sums (a part a warp) lie in Smem::o");
static_assert(2 * (sizeof(Smem<2, 1>) + 1024) <= 227 * 1024 && sizeof(Smem<2, 2>) <= 227 * 1024 - 1024,
              "two CTAs an SM, one with more than 8 heads a group");

template <typename T, int NQ, int HN, bool kTwice>
cudaError_t launch_t(const Attn4Args &A, int sms, cudaStream_t s) {
    auto kern = k_attn4<T, NQ, HN, kTwice>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<NQ, HN>));
    if (e != cudaSuccess) return e;
    // every CTA resident at once (no CTA waits for another, but equal runs should start together)
    const long long most = (long long)A.units * ((A.pool ? A.max_sel : 0) + (long long)(A.cache ? A.max_pages : 0));
    const long long runs = (most + (long long)A.units * kOver + kMinRun - 1) / kMinRun;
    const int ctas = Shape<HN>::kCtas * sms < max_ctas(sms) ? Shape<HN>::kCtas * sms : max_ctas(sms);
    const int grid = (int)(runs < ctas ? (runs > 0 ? runs : 1) : ctas);
    return launch_dependent(kern, dim3(grid), dim3(Shape<HN>::kThreads), sizeof(Smem<NQ, HN>), s, A);
}

}  // namespace

// SMs of the current device (asked of the driver once a device).
int device_sms() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    n = n > 0 ? n : 1;
    if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

size_t attn4_workspace(const ice_params &p) { return ws_layout(p, device_sms(), nullptr).bytes; }

cudaError_t launch_attn4(const ice_params &p, const void *Q, const void *records, const int32_t *page_len,
                         const int32_t *sel_pages, const int32_t *sel_count, int max_sel, const ice_cache4 *cache,
                         const int32_t *lens, float scale, float *O, float *lse, void *ws, int32_t *err,
                         cudaStream_t s) {
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
    A.g = p.n_q_heads / p.n_kv_heads, A.hq = p.n_q_heads, A.hkv = p.n_kv_heads, A.units = units_of(p);
    A.scale = scale;
    A.O = O, A.lse = lse, A.err = err;
    const int sms = device_sms();
    const Attn4Ws w = ws_layout(p, sms, ws);
    A.ticket = w.ticket, A.group_ticket = w.group_ticket, A.part_ml = w.part_ml, A.part_o = w.part_o;
    if (p.dtype == ICE_BF16)
        return A.g <= 4   ? launch_t<__nv_bfloat16, 1, 1, true>(A, sms, s)
               : A.g <= 8 ? launch_t<__nv_bfloat16, 1, 1, false>(A, sms, s)
                          : launch_t<__nv_bfloat16, 1, 2, false>(A, sms, s);
    return A.g <= 4   ? launch_t<float, 2, 1, true>(A, sms, s)
           : A.g <= 8 ? launch_t<float, 2, 1, false>(A, sms, s)
                      : launch_t<float, 2, 2, false>(A, sms, s);
}

}  // namespace ice
