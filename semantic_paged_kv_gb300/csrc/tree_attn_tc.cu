// Attention of drafted tokens over 4-bit pages on the tensor cores, for bf16
// rows: ice_cache4_attn_tree and ice_sparse_attn_tree4.
//   O[t] = sum_j exp(scale q_t . k_j) v_j / sum_j exp(scale q_t . k_j),
// j over the unit's pages, the ancestors of node t and t itself.
//
// The nodes of a tree share what they read: with T nodes and g heads a group
// T g query rows meet every key, so that the work is a matrix product (tcgen05)
// and the 4-bit pages are unpacked once for up to 128 rows.
//
// Roles in a CTA (20 warps, one CTA an SM):
//   10 warps unpack tiles of 128 tokens to fp16 in shared memory, page by page in
//     turn (K rows by token, V transposed: tokens are the contraction of the
//     second product), the next page on its way in their registers; three tiles
//     of K and of V;
//   2 threads issue the products, one S = Q K^T (128 x 128 x 128) of a tile, one O
//     += P V, with Q and P in tensor memory (operands from there leave shared
//     memory's bandwidth to K, V and the unpacking);
//   8 warps take the softmax, two threads a row, each half of a tile's tokens.
// Tensor memory: S of two tiles (128 columns each), O (128), Q and P (64 each).
//
// What bounds it: a tile costs an SM about 2200 clocks, the products 1024 of them.  Unpacking (a warp takes 2900 clocks a page;
// 10 of them 8 pages in 2300) and the softmax (2000 for a tile, two warps a scheduler) share the schedulers' issue; neither
// waits long for the other, and neither for memory.  10 unpacking warps leave 96 registers a thread: 8 take 136 us for 4 x 50k
// tokens of 64/8 heads and 16 nodes, 9 133, 10 126, 12 and 14 (80 registers) 139, 16 (72) 165.  Measured: that case 125 us
// (0.84 PFLOP/s, 1.8 TB/s), 16 x 100k 817 to 850 us (0.75 to 0.78), a chunk of 1000 tokens of 32/8 heads behind 36,864 693 us
// (0.88).  Short calls are bound by what a CTA does once (12,000 clocks before the first tile, 5,000 after the last), much of it the
// first pass through its code: loops that run once or twice are not unrolled (node rows: 9 sequences of 32 heads and one set of
// lengths 68 us, 83 unrolled by 4).
//
// Numbers: a code's value mid + step (c - 7.5) is rounded once, to fp16 (half a
// step, 2^-11, where the plain bf16 operand would lose 2^-9; elements below 2^-14,
// where fp16's steps stop shrinking, 2^-25, and so does a mid there), queries
// (bf16) are exact in fp16 after a power of two of their row.  Tokens whose |mid| + 7.5
// step lies outside 2^-4 .. 2^8 take a power of two of their own, which the
// softmax gives back: on scores for keys; for values on the weights, whose
// maximum is then kept apart from that of the sum, so that neither a large value
// of no weight costs others their bits nor a small one its own.  P is rounded to
// fp16, 2^6 above its running maximum's 1; that maximum only moves when a score
// passes it by 2^8 (O is scaled then).  Sums are fp32.
#include <cuda_fp16.h>
#include <float.h>

#include "tc_common.cuh"
#include "tree.cuh"

namespace ice {
namespace {

using namespace tree;
using namespace tc;

constexpr int kRows = kTreeRowsTc;
constexpr int kSoftWarps = 8, kLoadWarps = 10, kMmaWarp = kSoftWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 2);
constexpr int kStages = 3;
constexpr uint32_t kTileBytes = 128 * 128 * 2, kHalfBytes = kTileBytes / 2;
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColP = 448;
// A tile's Info is overwritten with K of the tile kInfos behind it, which waits for the scores of kStages tiles before
// that, which wait for the weights of two before those.
constexpr int kInfos = 8;
static_assert(32 * kSoftWarps == kMaxNodes, "a softmax thread a node");
static_assert(kInfos >= kStages + 2, "an Info outlives its softmax");
constexpr float kLazy = 8.f;  // powers of two that a score may pass the running maximum by
constexpr float kTop = 6.f;   // powers of two that P has above exp2(score - maximum)
// On a part's sum: without the power that weights can have, it is at most the number of the part's tokens, and the join's
// products of sums and values stay as small as the values allow.
constexpr float kPartSum = 0x1p-14f;
static_assert(kTop + kLazy == 14.f, "the largest weight");
constexpr float kMost = 16384.f;  // of the sum of a thread's weights of a tile (2^(kTop + kLazy)); above, the maximum moves
// kind::f16 instruction descriptor: D fp32, A and B fp16, both K-major, M = N = 128.
constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// What the softmax has to know of a tile.
struct Info {
    float kf[kTile];            // powers of two that K was divided by
    float vf[kTile];            // exponents of those of V
    uint16_t mask[kTilePages];  // used slots
    uint16_t odd[kTilePages];   // whether a page has a kf that is not 1 or a vf that is not 0
};
// A load warp's (step, mid) of 16 tokens in fp16.
struct MetaScratch {
    uint32_t k[16][4];     // 2^10 step and mid, each twice, of both groups
    uint16_t v[2][2][16];  // [group][2^10 step, mid][token]
};

struct Smem {
    unsigned char k[kStages][kTileBytes];
    unsigned char v[kStages][kTileBytes];
    Info info[kInfos];
    MetaScratch meta[kLoadWarps];
    Ancestors anc;
    float factor[kRows];       // of a segment's rows
    float2 split[kRows];       // the same as a product (score_of)
    float2 half[2][2][kRows];  // what the two threads of a row tell each other, in two tiles in turn
    PlanScratch plan;
    Args args;
    unsigned long long k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], s_ready[2], p_ready[2], q_full;
    unsigned long long drained[2];  // the products of the two issuing threads, after a wait that gave up
    uint32_t tmem;
    int bad;   // a node's value is not finite
    int dead;  // a wait gave up
    int seen;  // tiles whose scores are there
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "one CTA an SM");

// The CTA's shared memory, from the first 1024-byte boundary on (128-byte swizzled operands).
extern __shared__ unsigned char smem_raw[];
__device__ __forceinline__ Smem &shared() {
    return *reinterpret_cast<Smem *>(smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u));
}

// Barriers of the softmax threads: all of them, and the two threads of every row (warps w and w + 4).  Every softmax warp
// goes through the same segments and tiles, also after a wait has given up, so that all of them come here.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void pair_sync() {
    asm volatile("bar.sync %0, 64;" ::"r"(2 + (int)((threadIdx.x >> 5) & 3)) : "memory");
}
// The same, and whether x holds in all 64 threads.
__device__ __forceinline__ bool pair_all(bool x) {
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.red.and.pred q, %2, 64, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((int)x), "r"(2 + (int)((threadIdx.x >> 5) & 3))
        : "memory");
    return all != 0;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
// TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 16 rows (an eighth of the warps' 128) and 32 columns: lane l has columns 8 k + 2 (l % 4) and the next one of rows l / 4 (r[4
// k], r[4 k + 1]) and l / 4 + 8.
__device__ __forceinline__ void tmem_st_fragment(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tensor memory] (+)= A B with A in tensor memory.
__device__ __forceinline__ void umma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kIdesc), "r"(accumulate)
        : "memory");
}

// 16 fp32 TMEM columns of this thread's lane (no wait).
__device__ __forceinline__ void tmem_ld16f(uint32_t a, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(a));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// Two scores, x times a key's kf and its row's factor.  kf and the factor join first: a large key's power with the product, or
// a small query's with the scale, leaves fp32's range where the score does not.  Factors in 2^-100 .. 2 are safe as they are;
// one beyond, which may be no fp32 number itself, goes in two parts (kWide).  (x = 0: 0)
template <bool kWide> __device__ __forceinline__ float2 scores_of(float x0, float x1, float2 kf, float2 split) {
    const float2 k = upk2(mul2(pk2(kf.x, kf.y), pk2(split.y, split.y)));
    if (kWide) return make_float2(x0 * split.x * fminf(k.x, FLT_MAX), x1 * split.x * fminf(k.y, FLT_MAX));
    return upk2(mul2(pk2(x0, x1), pk2(k.x, k.y)));
}
// The factor |sl| 2^-e2 as (1, factor) where that is safe, otherwise with a power of two in 2^-126 .. 2^126 as the second part.
__device__ __forceinline__ float2 split_of(float sl, int e2) {
    const float f = fabsf(sl) * pow2(-e2);
    if (f >= 0x1p-100f && f <= 2.f) return make_float2(1.f, f);
    const int es = min(max((int)((__float_as_uint(sl) >> 23) & 255u) - 127, -126), 126), e = min(max(es - e2, -126), 126);
    return make_float2(fabsf(sl) * pow2(-es) * pow2(es - e2 - e), pow2(e));
}
// The exponent by whose power a token of largest element `big` is divided (0: none).
__device__ __forceinline__ int exponent_for(float big) {
    if ((big >= 0.0625f && big <= 256.f) || big == 0.f || !(big < INFINITY)) return 0;
    return min(max((int)((__float_as_uint(big) >> 23) & 255u) - 127, -126), 126);
}

// A run's tiles of one segment.
struct Piece {
    int i0, n, b, h, row0, rows;
    __device__ __forceinline__ Piece(const Args &A, const Segment &s, const Run &run) {
        i0 = (int)max(-s.first, 0ll);
        n = max((int)min((long long)s.n, run.n - s.first) - i0, 0);
        b = s.u / A.hkv, h = s.u - b * A.hkv;
        row0 = s.blk * kRows;
        rows = min(kRows, s.nodes * A.g - row0);
    }
};

__device__ __forceinline__ bool dead(const Smem &S) { return *static_cast<const volatile int *>(&S.dead) != 0; }
// A bounded wait; once one has given up, all do.
__device__ __forceinline__ bool wait_for(Smem &S, unsigned long long &bar, uint32_t parity) {
    if (mbar_test(&bar, parity)) return true;
    if (!dead(S) && mbar_wait(&bar, parity, S.args.fault ? kFaultWaitNs : kWaitNs)) return true;
    *static_cast<volatile int *>(&S.dead) = 1;
    set_err(S.args.err, ICE_ERR_TIMEOUT);
    return false;
}
// Waits until the scores of `tiles` tiles are there.  A wait on a phase's parity cannot tell a phase from the one two before: it
// is right where the waiting warp is at most a round of the ring ahead.  Warps without a slot in a segment (it has eight a
// tile) would pass over any number of short segments, so every segment begins with this.
__device__ __forceinline__ bool wait_seen(Smem &S, int tiles) {
    const volatile int &seen = S.seen;
    if (seen >= tiles) return true;
    const unsigned long long t0 = now_ns();
    while (!dead(S)) {
        if (seen >= tiles) return true;
        if (now_ns() - t0 > kWaitNs) break;
    }
    *static_cast<volatile int *>(&S.dead) = 1;
    set_err(S.args.err, ICE_ERR_TIMEOUT);
    return false;
}
// A tile's place in the rings (tiles of a CTA are counted over its segments) and the phase of its uses.
__device__ __forceinline__ uint32_t stage_of(uint32_t at) { return at % kStages; }
__device__ __forceinline__ uint32_t round_of(uint32_t at) { return at / kStages & 1; }

// ------------------------------------------------------------ load warps --
// Two codes of a word, c at bits 0 .. 3 of a half (c 2^-24 as fp16) or 4 .. 7 (c 2^-20), as (c - 7.5) 2^-10, exactly; times
// 2^10 step plus mid: rounded once.
__device__ __forceinline__ uint32_t low_pair(uint32_t w, uint32_t step, uint32_t mid) {
    return hfma2(hfma2(w & 0x000F000Fu, 0x74007400u, 0x9F809F80u), step, mid);
}
__device__ __forceinline__ uint32_t high_pair(uint32_t w, uint32_t step, uint32_t mid) {
    return hfma2(hfma2(w & 0x00F000F0u, 0x64006400u, 0x9F809F80u), step, mid);
}

struct Loader {
    const Args &A;
    Smem &S;
    const int lane, warp;  // warp of the load warps; it takes slots warp, warp + kLoadWarps, .. of a segment's tiles (a tile has 8)
    // the pages of its slots 32 j .., one a lane; and the page numbers of the next 32
    const unsigned char *page;
    int page_len, ahead, base, x0;

    __device__ __forceinline__ Loader(const Args &A, Smem &S, int warp) : A(A), S(S), lane(threadIdx.x & 31), warp(warp) {}

    __device__ __forceinline__ int place(int n) const { return x0 + (n + lane) * kLoadWarps + warp; }
    __device__ __forceinline__ void look_ahead(const Segment &s, int n) {
        const int x = place(n);
        ahead = -1;
        if (x < s.cnt.x)
            ahead = A.sel_pages[(size_t)s.u * A.max_sel + x];
        else if (x < pages_of(s.cnt))
            ahead = A.table[(size_t)(s.u / A.hkv) * A.max_pages + (x - s.cnt.x)];
    }
    // (the segment's tiles from `tile` on)
    __device__ __forceinline__ void start(const Segment &s, int tile) {
        x0 = tile * kTilePages;
        base = -1;
        look_ahead(s, 0);
    }
    // a page on its way (nothing of it waits)
    const unsigned char *rec;
    int live;        // used slots
    uint2 meta;      // (step, mid) of K (lanes 0 .. 15) or V (16 .. 31) of token lane % 16
    uint4 k[2];      // K: tokens 8 j + k_token(), words lane % 4 + 4 x
    uint2 v[4];      // V: pieces p and p + 8 of four token pairs (below)

    // The page of this warp's slot n; where there is none, some record (its codes meet steps of zero).
    __device__ __forceinline__ void find(const Segment &s, int n) {
        if (base != (n & ~31)) {  // 32 further pages, whose numbers have been on their way since the last time
            base = n & ~31;
            const int x = place(base), id = ahead;
            page = nullptr, page_len = 0;
            if (x < pages_of(s.cnt)) page = page_of_id(A, s.u, s.cnt, x, id, page_len);
            if (!page) page = A.cache ? A.cache : A.pool;
            look_ahead(s, base + 32);
        }
        rec = reinterpret_cast<const unsigned char *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(page), n & 31));
        live = __shfl_sync(0xffffffffu, page_len, n & 31);
        // the one after it into L2 (unless its number is still on its way): its loads then take half the time
        const unsigned char *after = reinterpret_cast<const unsigned char *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(page), (n + 1) & 31));
        if (((n + 1) & 31) && lane < q4::kRecord / 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(after + 128 * lane));
    }
    __device__ __forceinline__ void load_k() {
        meta = make_uint2(0u, 0u);
        if ((lane & 15) < live)
            meta = *reinterpret_cast<const uint2 *>(rec + (lane < 16 ? q4::kKMeta : q4::kVMeta) + (lane & 15) * 8);
        const uint4 *x = reinterpret_cast<const uint4 *>(rec) + 4 * k_token() + (lane & 3);
        k[0] = ld_stream16(x);
        k[1] = ld_stream16(x + 32);
    }
    __device__ __forceinline__ void load_v() {
        const uint2 *x = reinterpret_cast<const uint2 *>(rec + q4::kV) + v_half() * 64 + (v_piece() & 7) * 2 + (lane >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(x + 16 * i);
    }
    // A lane's V: pieces p and p + 8 (of one group) for 8 tokens, half of the page.  Of any 8 lanes that store together, the
    // piece's lowest bit, the half and which two of a piece's four elements come first differ, so that they reach all banks.
    __device__ __forceinline__ int v_half() const { return (lane >> 1) & 1; }
    __device__ __forceinline__ int v_piece() const { return (lane & 1) | ((lane >> 1) & 6) | (lane & 16); }

    // (step, mid): powers of two, operands, and what the softmax has to know.
    __device__ __forceinline__ void put_meta(int slot, Info &info) {
        MetaScratch &M = S.meta[warp];
        const int t = lane & 15;
        const float2 a = q4::unpack_meta(meta.x), c = q4::unpack_meta(meta.y);
        const int e = exponent_for(fmaxf(fabsf(a.y) + 7.5f * a.x, fabsf(c.y) + 7.5f * c.x));
        const float f = pow2(-e);  // (up to 2^126: 2^10 goes to the step)
        const uint32_t x = half2_of(a.x * f * 1024.f, a.y * f), y = half2_of(c.x * f * 1024.f, c.y * f);
        if (lane < 16) {
            *reinterpret_cast<uint4 *>(M.k[t]) = make_uint4(__byte_perm(x, x, 0x1010), __byte_perm(x, x, 0x3232),
                                                            __byte_perm(y, y, 0x1010), __byte_perm(y, y, 0x3232));
            info.kf[16 * slot + t] = pow2(e);
        } else {
            M.v[0][0][t] = (uint16_t)x, M.v[0][1][t] = (uint16_t)(x >> 16);
            M.v[1][0][t] = (uint16_t)y, M.v[1][1][t] = (uint16_t)(y >> 16);
            info.vf[16 * slot + t] = (float)e;
        }
        const bool odd = __any_sync(0xffffffffu, e != 0);
        if (lane == 0) info.mask[slot] = (uint16_t)((1u << live) - 1u), info.odd[slot] = odd;
        __syncwarp();
    }
    // K lanes: tokens four apart are neighbours, so that any 8 lanes that store together reach all banks.
    __device__ __forceinline__ int k_token() const { return (lane >> 3) | (lane & 4); }
    __device__ __forceinline__ void put_k(int slot, uint32_t dst) {
        const int i = lane & 3;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = 8 * j + k_token();
            const uint4 m = *reinterpret_cast<const uint4 *>(S.meta[warp].k[t]);
            const uint32_t row = dst + (16 * slot + t) * 128, a0 = row + ((i ^ (t & 7)) << 4), a1 = a0 ^ 64u;
            // word x: elements 8 (i + 4 x) .., in group x / 2
            put8(a0, k[j].x, m.x, m.y), put8(a1, k[j].y, m.x, m.y);
            put8(a0 + kHalfBytes, k[j].z, m.z, m.w), put8(a1 + kHalfBytes, k[j].w, m.z, m.w);
        }
    }
    __device__ __forceinline__ static void put8(uint32_t at, uint32_t w, uint32_t st, uint32_t md) {
        const uint32_t u = w >> 8;
        sts128(at, low_pair(w, st, md), high_pair(w, st, md), low_pair(u, st, md), high_pair(u, st, md));
    }
    __device__ __forceinline__ void put_v(int slot, uint32_t dst) {
        const uint16_t(&vm)[2][16] = S.meta[warp].v[lane >> 4];
        const uint4 st = *reinterpret_cast<const uint4 *>(&vm[0][8 * v_half()]);
        const uint4 md = *reinterpret_cast<const uint4 *>(&vm[1][8 * v_half()]);
        const int c = ((slot & 3) * 2 + v_half()) ^ (4 * (lane & 1)), flip = (lane >> 2) & 1;  // (d & 7 = 4 (p & 1) + e)
        const uint32_t base = dst + (slot >> 2) * kHalfBytes + 4 * v_piece() * 128;
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // the second piece is 32 elements further
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // elements e and e + 1 of the piece
                const int e = 2 * (x ^ flip), by = 4 * e;
                const uint32_t w0 = (y ? v[0].y : v[0].x) >> by, w1 = (y ? v[1].y : v[1].x) >> by;
                const uint32_t w2 = (y ? v[2].y : v[2].x) >> by, w3 = (y ? v[3].y : v[3].x) >> by;
                const uint32_t at = base + y * 32 * 128 + e * 128;
                sts128(at + ((c ^ e) << 4), low_pair(w0, st.x, md.x), low_pair(w1, st.y, md.y),
                       low_pair(w2, st.z, md.z), low_pair(w3, st.w, md.w));
                sts128(at + 128 + ((c ^ e ^ 1) << 4), high_pair(w0, st.x, md.x), high_pair(w1, st.y, md.y),
                       high_pair(w2, st.z, md.z), high_pair(w3, st.w, md.w));
            }
        }
    }

    // 16 of a tile's nodes: rows of 16 vectors of 8 elements, 16 lanes a row.
    __device__ __forceinline__ void node_k(uint32_t dst, int slot, const Segment &s, int b, int h, int j0, Info &info) {
        const int c = lane & 15;
        bool odd = false, bad = false;
        // the power of two of a row, from its finite elements (a key of infinities has a power of 1 at least: times a smaller one
        // and a small factor its scores would be 0 times infinity)
        auto power = [&](const float (&x)[8], float infinite) {
            float big = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : infinite);
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
            return exponent_for(big);
        };
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const int token = 16 * slot + 2 * i + (lane >> 4), node = j0 + token;
            if (j0 + 16 * slot + 2 * i >= s.nodes) {  // (its keys meet no row)
                if (c == 0) info.kf[token] = 1.f, info.vf[token] = 0.f;
                continue;
            }
            q4::Vec8<__nv_bfloat16> kk, vv;
            kk.zero(), vv.zero();
            if (node < s.nodes) {
                kk.load(row_ptr<__nv_bfloat16>(A.k, b, node, h) + 8 * c);
                vv.load(row_ptr<__nv_bfloat16>(A.v, b, node, h) + 8 * c);
            }
            float x[8], y[8];
            kk.get(x);
            vv.get(y);
            const int ek = power(x, 1.f), ev = power(y, 0.f);  // (the softmax needs V's with the scores, before V itself is put)
            const float f = pow2(-ek);
            sts128(dst + (c >> 3) * kHalfBytes + token * 128 + (((c & 7) ^ (token & 7)) << 4),
                   half2_of(x[0] * f, x[4] * f), half2_of(x[1] * f, x[5] * f), half2_of(x[2] * f, x[6] * f),
                   half2_of(x[3] * f, x[7] * f));
            if (c == 0) info.kf[token] = pow2(ek), info.vf[token] = (float)ev;
            odd |= ek != 0 || ev != 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) bad |= !(fabsf(y[e]) < INFINITY);
        }
        odd = __any_sync(0xffffffffu, odd);
        if (bad) S.bad = 1;
        if (lane == 0) info.odd[slot] = odd;
    }
    __device__ __forceinline__ void node_v(uint32_t dst, int slot, const Segment &s, int b, int h, int j0, const Info &info) {
        const int c = lane & 15;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const int token = 16 * slot + 4 * i + 2 * (lane >> 4), node = j0 + token;  // and the next one
            float x[8], y[8];
            q4::Vec8<__nv_bfloat16> w, z;
            w.zero(), z.zero();
            if (node < s.nodes) w.load(row_ptr<__nv_bfloat16>(A.v, b, node, h) + 8 * c);
            if (node + 1 < s.nodes) z.load(row_ptr<__nv_bfloat16>(A.v, b, node + 1, h) + 8 * c);
            w.get(x);
            z.get(y);
            const float fx = pow2(-(int)info.vf[token]), fy = pow2(-(int)info.vf[token + 1]);
            const uint32_t base = dst + (token >> 6) * kHalfBytes + (token & 7) * 2;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = 8 * c + e;
                const float a = fabsf(x[e]) < INFINITY ? x[e] * fx : 0.f, g = fabsf(y[e]) < INFINITY ? y[e] * fy : 0.f;
                sts32(base + d * 128 + ((((token & 63) >> 3) ^ (d & 7)) << 4), half2_of(a, g));
            }
        }
    }
};

// ICE_FAULT's timeout: the keys of this warp's first slot and nothing else, so that products of scores are issued and values
// never arrive.  (Apart: a test of the flag in the loop below costs a chunk of 1000 behind 36k 2%.)
__device__ __noinline__ void unpack_first_keys(const Run run) {
    Smem &S = shared();
    const Args &A = S.args;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kSoftWarps;
    const Segment &seg = S.plan.seg;
    const Piece P(A, seg, run);
    if (w >= kTilePages || P.n == 0) return;
    Loader L(A, S, w);
    if (P.i0 < seg.n_page) {
        L.start(seg, P.i0);
        L.find(seg, 0);
        L.load_k();
        L.put_meta(w, S.info[0]);
        L.put_k(w, su32(S.k[0]));
    } else {
        L.node_k(su32(S.k[0]), w, seg, P.b, P.h, (P.i0 - seg.n_page) * kTile, S.info[0]);
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.k_full[0]);
}

// The load warps' part: the run's tiles, one after another.  (The roles are not inlined: each has its own registers.)
__device__ __noinline__ void unpack_tiles(const Run run) {
    Smem &S = shared();
    const Args &A = S.args;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kSoftWarps;
    Loader L(A, S, w);
    uint32_t tile0 = 0;
    Segment seg = S.plan.seg;
    for (;; next_segment<kRows>(A, seg)) {
        if (seg.first >= run.n) return;
        const Piece P(A, seg, run);
        if (P.n == 0) continue;
        const int slots = P.n * kTilePages, pages = min(max(seg.n_page - P.i0, 0) * kTilePages, slots);
        // slot x: its keys as soon as the stage is free of those of kStages tiles before, then its values
        int x = w;
        auto slot_at = [&] { return x % kTilePages; };
        auto tile_at = [&] { return tile0 + x / kTilePages; };
        auto begin = [&](unsigned long long (&empty)[kStages]) {
            return wait_for(S, empty[stage_of(tile_at())], round_of(tile_at()) ^ 1);
        };
        auto end = [&](unsigned long long (&full)[kStages]) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage_of(tile_at())]);
        };
        L.start(seg, P.i0);
        if (x < pages) {
            L.find(seg, 0);
            L.load_k();
            L.load_v();
        }
        if (!wait_seen(S, (int)tile0 - kStages + 1)) return;
        for (int n = 1; x < pages; ++n) {
            const int slot = slot_at(), next = x + kLoadWarps;
            const uint32_t at = tile_at();
            if (!begin(S.k_empty)) return;
            L.put_meta(slot, S.info[at & (kInfos - 1)]);
            L.put_k(slot, su32(S.k[stage_of(at)]));
            end(S.k_full);
            if (next < pages) {  // (the next page's loads as soon as their registers are free)
                L.find(seg, n);
                L.load_k();
            }
            if (!begin(S.v_empty)) return;
            L.put_v(slot, su32(S.v[stage_of(at)]));
            end(S.v_full);
            if (next < pages) L.load_v();
            x = next;
        }
        for (; x < slots; x += kLoadWarps) {
            Info &info = S.info[tile_at() & (kInfos - 1)];
            const int j0 = (P.i0 + x / kTilePages - seg.n_page) * kTile;
            if (!begin(S.k_empty)) return;
            L.node_k(su32(S.k[stage_of(tile_at())]), slot_at(), seg, P.b, P.h, j0, info);
            end(S.k_full);
            if (!begin(S.v_empty)) return;
            L.node_v(su32(S.v[stage_of(tile_at())]), slot_at(), seg, P.b, P.h, j0, info);
            end(S.v_full);
        }
        tile0 += P.n;
        if (seg.end() >= run.n) return;
    }
}

// --------------------------------------------------------------- products --
// What step kk of 16 adds to an operand's descriptor.
__device__ __forceinline__ uint32_t step_at(uint32_t kk) { return (kk >> 2) * (kHalfBytes >> 4) + (kk & 3) * 2; }
__device__ __forceinline__ void product(uint32_t d, uint32_t a, const void *b, bool add) {
    const uint64_t desc = sw128_desc(su32(b));
#pragma unroll
    for (uint32_t kk = 0; kk < 8; ++kk) umma_ta(d, a + 8 * kk, desc + step_at(kk), add || kk > 0);
}

// The products of the run's tiles: S by one thread, O by another, so that neither waits with the other's operands there.
template <bool kScores> __device__ __noinline__ void issue_products(const Run run, uint32_t tmem) {
    Smem &S = shared();
    const Args &A = S.args;
    uint32_t at = 0, n_seg = 0;
    Segment seg = S.plan.seg;
    for (;; next_segment<kRows>(A, seg)) {
        if (seg.first >= run.n) return;
        const Piece P(A, seg, run);
        if (P.n == 0) continue;
        if (kScores && !wait_for(S, S.q_full, n_seg++ & 1)) return;
        for (int i = 0; i < P.n; ++i, ++at) {
            const uint32_t stage = stage_of(at), half = at & 1, turn = at >> 1 & 1;
            if (kScores) {
                // (its scores' place has been read: the weights of two tiles before are there)
                if (!wait_for(S, S.k_full[stage], round_of(at)) || !wait_for(S, S.p_ready[half], turn ^ 1)) return;
                fence_after();
                product(tmem + kColS + 128 * half, tmem + kColQ, S.k[stage], false);
                umma_commit(&S.s_ready[half]);
                umma_commit(&S.k_empty[stage]);
            } else {
                if (!wait_for(S, S.v_full[stage], round_of(at)) || !wait_for(S, S.p_ready[half], turn)) return;
                fence_after();
                product(tmem + kColO, tmem + kColP, S.v[stage], i > 0);
                umma_commit(&S.v_empty[stage]);
            }
        }
        if (seg.end() >= run.n) return;
    }
}

// -------------------------------------------------------- softmax threads --
struct Row {
    float m, mo, l, r;  // running maxima of the scores (of the sum, of O), sum (of this thread's tokens), factor (> 0)
};

// Scales this thread's 64 elements of O by f (a warp at a time).
__device__ __forceinline__ void scale_o(uint32_t at, float f) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        float x[16];
        uint32_t y[16];
        tmem_ld16f(at + 16 * c, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i] * f);
        tmem_st16(at + 16 * c, y);
    }
    tmem_wait_st();
}

// New maximum of a row and O's factor; whether O of the warp has to be scaled.
__device__ __forceinline__ bool raise(float &m, float top, bool first, float &f) {
    f = 1.f;
    if (first) {
        m = fmaxf(top, -FLT_MAX);
        return false;
    }
    const bool up = top > m + kLazy || (m == -FLT_MAX && top > m);
    if (up) f = exp2_fast(m - top), m = top;
    return __any_sync(0xffffffffu, up);
}

// Row's bits of the 64 nodes from j0 on.
__device__ __forceinline__ uint2 node_mask(const Smem &S, bool tree, int node, int j0) {
    uint32_t mask[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (tree) {
            mask[c] = S.anc.mask[node][(j0 >> 5) + c];
        } else {
            const int n = node - (j0 + 32 * c) + 1;
            mask[c] = n >= 32 ? 0xffffffffu : (n > 0 ? (1u << n) - 1u : 0u);
        }
    }
    return make_uint2(mask[0], mask[1]);
}

// The weights of this thread's 64 scores and their sum.  Columns are loaded ahead while others are worked on.
struct Scores {
    uint32_t s_at, p_at, mask[2];
    __device__ __forceinline__ void seen(int c, float (&x)[16]) const {
        const uint32_t w = (c < 2 ? mask[0] : mask[1]) >> (16 * (c & 1));
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = w >> i & 1u ? x[i] : -INFINITY;
    }
    __device__ __forceinline__ float largest() const {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float x[16];
            tmem_ld16f(s_at + 16 * c, x);
            tmem_wait_ld();
            seen(c, x);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                top[0] = max3(top[0], x[i], x[i + 1]), top[1] = max3(top[1], x[i + 2], x[i + 3]);
        }
        return fmaxf(top[0], top[1]);
    }
    // exp2(score r + off), and their sum
    template <bool kMask> __device__ __forceinline__ float weights(float r, float off, uint32_t (&w)[2][16]) const {
        const unsigned long long r2 = pk2(r, r), off2 = pk2(off, off);
        unsigned long long sum[2] = {0ull, 0ull};
        float s[2][16];
        tmem_ld16f(s_at, s[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            tmem_wait_ld();
            if (c < 3) tmem_ld16f(s_at + 16 * (c + 1), s[(c + 1) & 1]);
            float(&x)[16] = s[c & 1];
            if (kMask) seen(c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = upk2(fma2(pk2(x[2 * i], x[2 * i + 1]), r2, off2));
                const float a = exp2_fast(y.x), b = exp2_fast(y.y);
                sum[i & 1] = add2(sum[i & 1], pk2(a, b));
                w[c >> 1][8 * (c & 1) + i] = half2_of(a, b);
            }
        }
        const float2 t = upk2(add2(sum[0], sum[1]));
        return t.x + t.y;
    }
    __device__ __forceinline__ void store(const uint32_t (&w)[2][16]) const {
        tmem_st16(p_at, w[0]);
        tmem_st16(p_at + 16, w[1]);
    }
    // The same where keys or values carry powers of two of their own, or the two maxima have parted.  (Packed pairs: 4 x 50k
    // tokens that all have powers of their own take 303 us, one score after another 325 to 377 by the order of the factors.)
    template <bool kWide> __device__ __forceinline__ float2 largest_any(const float *kf, const float *vf, float2 split) const {
        float top = -INFINITY, top_o = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float x[16];
            tmem_ld16f(s_at + 16 * c, x);
            tmem_wait_ld();
            const uint32_t w = (c < 2 ? mask[0] : mask[1]) >> (16 * (c & 1));
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float2 y = scores_of<kWide>(x[i], x[i + 1], *reinterpret_cast<const float2 *>(kf + 16 * c + i), split);
                y.x = w >> i & 1u ? y.x : -INFINITY, y.y = w >> (i + 1) & 1u ? y.y : -INFINITY;
                const float2 e = *reinterpret_cast<const float2 *>(vf + 16 * c + i);
                const float2 z = upk2(add2(pk2(y.x, y.y), pk2(e.x, e.y)));
                top = max3(top, y.x, y.y), top_o = max3(top_o, z.x, z.y);
            }
        }
        return make_float2(top, top_o);
    }
    template <bool kWide>
    __device__ __forceinline__ float weights_any(const float *kf, const float *vf, float2 split, float off, float off_o) const {
        const unsigned long long off2 = pk2(off, off), off_o2 = pk2(off_o, off_o);
        unsigned long long sum = 0ull;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float x[16];
            uint32_t p[8];
            tmem_ld16f(s_at + 16 * c, x);
            tmem_wait_ld();
            const uint32_t w = (c < 2 ? mask[0] : mask[1]) >> (16 * (c & 1));
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float2 y = scores_of<kWide>(x[i], x[i + 1], *reinterpret_cast<const float2 *>(kf + 16 * c + i), split);
                y.x = w >> i & 1u ? y.x : -INFINITY, y.y = w >> (i + 1) & 1u ? y.y : -INFINITY;
                const float2 e = *reinterpret_cast<const float2 *>(vf + 16 * c + i);
                const unsigned long long y2 = pk2(y.x, y.y);
                const float2 a = upk2(add2(y2, off2)), z = upk2(add2(add2(y2, pk2(e.x, e.y)), off_o2));
                sum = add2(sum, pk2(exp2_fast(a.x), exp2_fast(a.y)));
                p[i >> 1] = half2_of(exp2_fast(z.x), exp2_fast(z.y));
            }
            tmem_st8(p_at + 8 * c, p);
        }
        const float2 t = upk2(sum);
        return t.x + t.y;
    }
};

// A segment's tiles (the CTA's tiles from tile0 on, the first n_page of pages), by the 256 softmax threads: thread (row,
// half).
__device__ __noinline__ Row soften_tiles(uint32_t tmem, uint32_t tile0, int n, int n_page, int node, float factor, int rows) {
    Smem &S = shared();
    const int warp = threadIdx.x >> 5, row = threadIdx.x & 127, hf = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t o_at = tmem + lanes + kColO + 64 * hf;
    Row R;
    R.m = R.mo = -FLT_MAX, R.l = 0.f, R.r = factor;
    for (int i = 0; i < n; ++i) {
        const uint32_t at = tile0 + i;
        wait_for(S, S.s_ready[at & 1], at >> 1 & 1);
        if (threadIdx.x == 0) *static_cast<volatile int *>(&S.seen) = (int)at + 1;
        __syncwarp();
        fence_after();
        if ((row & ~31) >= rows) {  // no row of this warp (and its partner): its rows of P and O mean nothing
            fence_before();
            if ((threadIdx.x & 31) == 0) mbar_arrive(&S.p_ready[at & 1]);
            continue;
        }
        const Info &info = S.info[at & (kInfos - 1)];
        const uint2 mask = i < n_page ? *reinterpret_cast<const uint2 *>(&info.mask[4 * hf])
                                      : node_mask(S, S.args.parents != nullptr, node, (i - n_page) * kTile + 64 * hf);
        const uint4 odd = *reinterpret_cast<const uint4 *>(info.odd);
        const Scores X{tmem + lanes + kColS + 128 * (at & 1) + 64 * hf, tmem + lanes + kColP + 32 * hf, {mask.x, mask.y}};
        const bool full = __all_sync(0xffffffffu, (mask.x & mask.y) == 0xffffffffu);
        const bool apart = __any_sync(0xffffffffu, (odd.x | odd.y | odd.z | odd.w) != 0u || !(R.m == R.mo));
        // P's place has been read, and O is that of the tile before
        auto o_done = [&] {
            if (i > 0) wait_for(S, S.v_empty[stage_of(at - 1)], round_of(at - 1));
            __syncwarp();
            fence_after();
        };
        // Against the maximum as it is first: weights that would be too large for fp16 show in their sum.
        bool done = false;
        if (i > 0 && !apart) {
            uint32_t w[2][16];
            const float l = full ? X.weights<false>(R.r, kTop - R.m, w) : X.weights<true>(R.r, kTop - R.m, w);
            done = pair_all(l <= kMost);
            if (done) {
                R.l += l;
                o_done();
                X.store(w);
            }
        } else if (i > 0) {
            // (so that both warps of a row come to the same barriers whatever they have read: after a wait that gave up a tile's
            // Info may still be written, and `apart` differ)
            pair_all(false);
        }
        if (!done) {
            // the row's maximum: that of its two threads
            float2 split = make_float2(1.f, 1.f);
            if (apart) split = S.split[row];
            const bool wide = __any_sync(0xffffffffu, split.x != 1.f);
            const float *kf = &info.kf[64 * hf], *vf = &info.vf[64 * hf];
            float2 top = !apart ? make_float2(X.largest() * R.r, 0.f)
                         : wide ? X.largest_any<true>(kf, vf, split) : X.largest_any<false>(kf, vf, split);
            S.half[at & 1][hf][row] = top;
            pair_sync();
            const float2 other = S.half[at & 1][hf ^ 1][row];
            top.x = fmaxf(top.x, other.x);
            top.y = apart ? fmaxf(top.y, other.y) : top.x;
            float f, fo;
            if (raise(R.m, top.x, i == 0, f)) R.l *= f;
            const bool up_o = raise(R.mo, top.y, i == 0, fo);
            o_done();
            if (up_o) scale_o(o_at, fo);
            if (apart) {
                R.l += wide ? X.weights_any<true>(kf, vf, split, kTop - R.m, kTop - R.mo)
                            : X.weights_any<false>(kf, vf, split, kTop - R.m, kTop - R.mo);
            } else {
                uint32_t w[2][16];
                R.l += X.weights<true>(R.r, kTop - R.m, w);
                X.store(w);
            }
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&S.p_ready[at & 1]);
    }
    return R;
}

// The queries of a segment into tensor memory, exact in fp16 after a power of two of the row; the factor of this thread's
// row's products.  Four lanes take a row of 16 (a row of the store's fragment) and read 64 bytes of it together.
__device__ __forceinline__ float put_queries(Smem &S, const Piece &P, uint32_t q_at) {
    const Args &A = S.args;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane & 3, row = threadIdx.x & 127;
    const int first = 32 * (warp & 3) + 16 * (warp >> 2) + (lane >> 2);  // and the one eight behind
    uint4 v[2][4];  // pieces 4 m + 2 (j % 2) + j / 2 of 8 elements
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = P.row0 + first + 8 * i, node = at / A.g;
        const uint4 *src = reinterpret_cast<const uint4 *>(row_ptr<__nv_bfloat16>(A.q, P.b, node, P.h * A.g + at - node * A.g));
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            v[i][m] = make_uint4(0u, 0u, 0u, 0u);
            if (first + 8 * i < P.rows) v[i][m] = src[4 * m + 2 * (j & 1) + (j >> 1)];
        }
    }
    const float sl = fminf(fmaxf(A.scale * 1.4426950408889634f, -FLT_MAX), FLT_MAX);
    float up[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t big2 = 0u;  // magnitudes: bf16 values in the order of their bits
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            big2 = __vmaxu2(big2, __vmaxu2(v[i][m].x & 0x7FFF7FFFu, v[i][m].y & 0x7FFF7FFFu));
            big2 = __vmaxu2(big2, __vmaxu2(v[i][m].z & 0x7FFF7FFFu, v[i][m].w & 0x7FFF7FFFu));
        }
        big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 1));
        big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 2));
        const uint32_t big = max(big2 & 0xFFFFu, big2 >> 16);
        const int e2 = min(max(14 - ((int)(big >> 7) - 127), -113), 126);
        up[i] = sl == 0.f ? 0.f : copysignf(pow2(e2), sl);
        const float f = sl == 0.f ? 1.f : fabsf(sl) * pow2(-e2);
        // (never zero: slots that are not seen have a score of -inf.  It counts where all of a tile's keys have powers of 1:
        // products are below 2^31 then, and scores with a factor below FLT_MIN as good as 0)
        if (j == 0) {
            const float nan = __int_as_float(0x7fc00000);
            const float2 split = split_of(sl, e2);
            S.factor[first + 8 * i] = big < 0x7F80u ? fminf(fmaxf(f, FLT_MIN), FLT_MAX) : nan;
            S.split[first + 8 * i] = make_float2(big < 0x7F80u ? split.x : nan, split.y);
        }
    }
    const bool odd = j & 1;
#pragma unroll
    for (int m = 0; m < 4; m += 2) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 y = v[i][m + x];
                auto lo = [&](uint32_t z) { return __uint_as_float(z << 16) * up[i]; };
                auto hi = [&](uint32_t z) { return __uint_as_float(z & 0xFFFF0000u) * up[i]; };
                // elements e and e + 4 side by side (the order of K's); the lane beside has the other half of both pieces
                const uint32_t a0 = half2_of(lo(y.x), lo(y.z)), a1 = half2_of(hi(y.x), hi(y.z));
                const uint32_t b0 = half2_of(lo(y.y), lo(y.w)), b1 = half2_of(hi(y.y), hi(y.w));
                const uint32_t r0 = __shfl_xor_sync(0xffffffffu, odd ? a0 : b0, 1);
                const uint32_t r1 = __shfl_xor_sync(0xffffffffu, odd ? a1 : b1, 1);
                w[8 * x + 2 * i] = odd ? r0 : a0, w[8 * x + 2 * i + 1] = odd ? r1 : a1;
                w[8 * x + 4 + 2 * i] = odd ? b0 : r0, w[8 * x + 4 + 2 * i + 1] = odd ? b1 : r1;
            }
        }
        tmem_st_fragment(q_at + ((uint32_t)(warp >> 2) << 20) + 16 * m, w);
    }
    tmem_wait_st();
    pair_sync();
    return S.factor[row];
}

// The softmax threads' part; the segment that starts here and goes on in other CTAs.
__device__ __noinline__ Part soften(const Run run, uint32_t tmem) {
    Smem &S = shared();
    const Args &A = S.args;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127, hf = warp >> 2, g = A.g;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    Part part{};
    uint32_t tile0 = 0;
    int anc_b = -1;
    Segment seg = S.plan.seg;
    for (;; next_segment<kRows>(A, seg)) {
        if (seg.first >= run.n) break;
        const Piece P(A, seg, run);
        if (P.n == 0) continue;  // (its tiles lie in the runs before)
        const bool out = row < P.rows;
        const int at_row = P.row0 + min(row, P.rows - 1), node = at_row / g, head = P.h * g + at_row % g;
        const bool tree = A.parents && P.i0 + P.n > seg.n_page && anc_b != P.b;
        const int up = tree && (int)threadIdx.x < seg.nodes ? A.parents[(size_t)P.b * A.n_nodes + threadIdx.x] : -1;
        const float factor = put_queries(S, P, tmem + lanes + kColQ);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.q_full);
        if (tree) {
            soft_sync();  // (the last ones have been read)
            find_ancestors(up, seg.nodes, S.anc, A.err, threadIdx.x, [] { soft_sync(); });
            anc_b = P.b;
        }
        Row R = soften_tiles(tmem, tile0, P.n, seg.n_page - P.i0, node, factor, P.rows);
        tile0 += P.n;
        // ---- the row's result, O / l
        const int free = tile0 & 1;  // (the last tile's side may still be read; the one before it not)
        S.half[free][hf][row].x = R.l;
        pair_sync();
        R.l = S.half[free][0][row].x + S.half[free][1][row].x;
        pair_sync();
        wait_for(S, S.v_empty[stage_of(tile0 - 1)], round_of(tile0 - 1));
        __syncwarp();
        fence_after();
        const bool whole = seg.first >= 0 && seg.end() <= run.n;
        if (!whole && seg.first >= 0) part = part_of<kRows>(seg, run, g);
        const size_t slot = (size_t)blockIdx.x * 2 + (seg.first > 0 ? 1 : 0);
        if (dead(S)) R.l = __int_as_float(0x7fc00000);  // a wait gave up: NaN
        const float none = whole ? __int_as_float(0x7fc00000) : 0.f;  // (all scores -inf; in a part: nothing seen)
        const float inv = 1.f / R.l, f = exp2_fast(0.5f * (R.mo - R.m));
        if (out && !whole && hf == 0) A.part_ml[slot * kPartRows + row] = make_float2(R.m, R.l * kPartSum);
        __nv_bfloat16 *dst = row_out<__nv_bfloat16>(A.o, P.b, node, head) + 64 * hf;
        const int nodes0 = max(P.i0 - seg.n_page, 0) * kTile, nodes1 = min((P.i0 + P.n - seg.n_page) * kTile, seg.nodes);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float x[16];
            tmem_ld16f(tmem + lanes + kColO + 64 * hf + 16 * c, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = R.l == 0.f ? none : x[i] * inv * f * f;
            if (S.bad) {  // infinities and NaN of the nodes that this row sees
#pragma unroll 1
                for (int j = nodes0; j < nodes1; ++j) {
                    const bool sees = A.parents ? S.anc.mask[node][j >> 5] >> (j & 31) & 1u : j <= node;
                    if (!sees) continue;
                    const __nv_bfloat16 *v = row_ptr<__nv_bfloat16>(A.v, P.b, j, P.h) + 64 * hf + 16 * c;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float y = __bfloat162float(v[i]);
                        if (!(fabsf(y) < INFINITY)) x[i] += y;
                    }
                }
            }
            if (out && whole) {
                store8<__nv_bfloat16>(dst + 16 * c, reinterpret_cast<const float(&)[8]>(x[0]));
                store8<__nv_bfloat16>(dst + 16 * c + 8, reinterpret_cast<const float(&)[8]>(x[8]));
            } else if (out) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    A.part_o[part_at(slot, 16 * hf + 4 * c + i, row)] =
                        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
            __syncwarp();
        }
        fence_before();
        if (seg.end() >= run.n) break;
    }
    return part;
}

__global__ void __launch_bounds__(kThreads, 1) k_tree_tc(const __grid_constant__ Args A) {
    Smem &S = shared();
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&S.k_full[i], kTilePages), mbar_init(&S.k_empty[i], 1);
            mbar_init(&S.v_full[i], kTilePages), mbar_init(&S.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&S.s_ready[i], 1), mbar_init(&S.p_ready[i], kSoftWarps);
        mbar_init(&S.q_full, kSoftWarps), mbar_init(&S.drained[0], 1), mbar_init(&S.drained[1], 1);
        mbar_init_fence();
        S.dead = 0, S.seen = 0, S.bad = 0, S.args = A;
    }
    if (warp == 0) tmem_alloc(&S.tmem, 512);
    dep_wait();
    const Run run = plan_run<kRows, kThreads>(A, S.plan);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = S.tmem;
    Part part{};
    if (run.n > 0) {
        if (warp < kSoftWarps)
            part = soften(run, tmem);
        else if (warp < kMmaWarp)
            S.args.fault ? unpack_first_keys(run) : unpack_tiles(run);
        else if (tid == 32 * kMmaWarp)
            issue_products<true>(run, tmem);
        else if (tid == 32 * kMmaWarp + 32)
            issue_products<false>(run, tmem);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    // Drain: after a wait that gave up, products may be under way that nobody waited for; they end before tensor memory is freed
    // and the CTA leaves (without one, the last segment's results have waited for all of them).
    if (dead(S)) {  // (the same for the whole CTA: nobody waits any more)
        const int issuer = (warp - kMmaWarp) & 1;
        if (warp >= kMmaWarp && (tid & 31) == 0) {
            umma_commit(&S.drained[issuer]);
            mbar_wait(&S.drained[issuer], 0);
        }
        __syncwarp();
        __syncthreads();
    }
    if (tid == 0) A.parts[blockIdx.x] = part;
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_tree_tc(const Args &A, int grid, cudaStream_t s) {
    const int smem = (int)sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_tree_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_tree_tc, dim3(grid), dim3(kThreads), smem, s, A);
}

}  // namespace ice
