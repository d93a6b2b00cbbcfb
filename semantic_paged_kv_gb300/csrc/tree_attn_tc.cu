// Attention of drafted tokens over 4-bit pages on the tensor cores, for bf16
// rows: ice_cache4_attn_tree and ice_sparse_attn_tree4.
//   O[t] = sum_j exp(scale q_t . k_j) v_j / sum_j exp(scale q_t . k_j),
// j over the unit's pages, the ancestors of node t and t itself.
//
// The nodes of a tree share what they read: with T nodes and g heads a group
// T g query rows meet every key, so that the work is a matrix product (tcgen05)
// and the 4-bit pages are unpacked once for up to 256 rows.
//
// Roles in a CTA (13 warps, one CTA an SM):
//   4 warps unpack a tile of 128 tokens to fp16 in shared memory (K rows by
//     token, V transposed: tokens are the contraction of the second product);
//   1 thread issues the products: S = Q K^T (128 x 128 x 128) and O += P V with
//     P in tensor memory;
//   2 x 4 warps take the softmax, a thread a row: two streams, so that the
//     products of one run beside the softmax of the other.  More than 128 rows:
//     a stream has 128 of them and all tiles; else both have the same rows and
//     every other tile, and are joined at the end.
// Tensor memory: S of both streams (128 columns each, P takes its first 64),
// O of both.
//
// Numbers: a code's value mid + step (c - 7.5) is rounded once, to fp16 (half a
// step, 2^-11, where the plain bf16 operand would lose 2^-9), queries (bf16) are
// exact in fp16 after a power of two of their row.  Tokens whose |mid| + 7.5
// step lies outside 2^-4 .. 2^15 take a power of two of their own, which the
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

constexpr int kRows = 128;  // of a stream
constexpr int kSoftWarps = 8, kLoadWarps = 4, kMmaWarp = kSoftWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr uint32_t kTileBytes = 128 * 128 * 2, kHalfBytes = kTileBytes / 2;
constexpr uint32_t kColS = 0, kColO = 256;  // of stream 0; stream 1's are 128 columns further
constexpr int kInfos = 4;
constexpr float kLazy = 8.f;  // powers of two that a score may pass the running maximum by
constexpr float kTop = 6.f;   // powers of two that P has above exp2(score - maximum)
// kind::f16 instruction descriptor: D fp32, A and B fp16, both K-major, M = N = 128.
constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// What the softmax has to know of a tile.
struct Info {
    float kf[kTile];    // powers of two that K was divided by
    float vf[kTile];    // exponents of those of V
    uint32_t mask[4];   // used slots
    uint32_t flags[4];  // of 32 tokens: 1: a kf is not 1, 2: a vf is not 0
};
// A load warp's (step, mid) of 32 tokens in fp16.
struct MetaScratch {
    uint32_t k[32][2];       // (step, mid) of both groups
    uint16_t v[2][2][2][16];  // [page][group][step, mid][token]
};

struct Smem {
    unsigned char q[2][kTileBytes];
    unsigned char k[2][kTileBytes];
    unsigned char v[2][kTileBytes];
    Info info[kInfos];
    MetaScratch meta[kLoadWarps];
    Ancestors anc;
    float2 join_ml[kRows];
    PlanScratch plan;
    unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2], s_ready[2], p_ready[2], q_full, o_ready, seg_done, soft;
    uint32_t tmem;
    int bad;   // a node's value is not finite
    int dead;  // a wait gave up
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "one CTA an SM");

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
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
// 16 (32) TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
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

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The exponent by whose power a token of largest element `big` is divided (0: none).
__device__ __forceinline__ int exponent_for(float big) {
    if ((big >= 0.0625f && big <= 32768.f) || big == 0.f || !(big < INFINITY)) return 0;
    return min(max((int)((__float_as_uint(big) >> 23) & 255u) - 127, -126), 126);
}

// A run's tiles of one segment.
struct Piece {
    int i0, n, b, h, row0, rows;
    bool wide;  // more than 128 rows: a stream has its own
    __device__ __forceinline__ Piece(const Args &A, const Segment &s, const Run &run) {
        i0 = (int)max(-s.first, 0ll);
        n = max((int)min((long long)s.n, run.n - s.first) - i0, 0);
        b = s.u / A.hkv, h = s.u - b * A.hkv;
        row0 = s.blk * kTreeRowsTc;
        rows = (int)min((long long)kTreeRowsTc, (long long)s.nodes * A.g - row0);
        wide = rows > kRows;
    }
};

// ------------------------------------------------------------ load warps --
// Eight codes of a word (c at bits 4 .. 7 of a half is 64 + c as fp16) times step plus mid: elements (0, 4), (1, 5), ..
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int e) {
    return hadd2(((e == 0 ? w << 4 : w >> (4 * e - 4)) & 0x00F000F0u) | 0x54005400u, 0xD478D478u);  // - 71.5
}

struct Loader {
    const Args &A;
    Smem &S;
    const int lane, warp;  // warp of the load warps
    uint4 k[4];            // K: page j / 2, tokens 8 (j % 2) + lane / 4, words 4 (lane % 4) ..
    uint32_t v[16];        // V: this lane's page, pieces and token pairs (below)
    uint2 mk, mv;          // (step, mid) of token `lane` of the two pages
    int live;              // used slots of its page
    // pages looked up: this warp's two pages of 16 tiles, one a lane
    const unsigned char *page;
    int page_len, looked;

    __device__ __forceinline__ Loader(const Args &A, Smem &S, int warp) : A(A), S(S), lane(threadIdx.x & 31), warp(warp) {}

    __device__ __forceinline__ void start(const Segment &s) { looked = -1; }
    __device__ __forceinline__ void look(const Segment &s, int tile) {
        const int base = tile & ~15;
        if (base == looked) return;
        looked = base;
        const int x = (base + (lane >> 1)) * kTilePages + 2 * warp + (lane & 1);
        page = nullptr, page_len = 0;
        if (x < pages_of(s.cnt)) page = page_at(A, s.u, s.cnt, x, page_len);
    }
    __device__ __forceinline__ const unsigned char *page_of(int tile, int j) {
        const int src = ((tile & 15) << 1) + j;
        return reinterpret_cast<const unsigned char *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(page), src));
    }
    __device__ __forceinline__ int len_of(int tile, int j) {
        return __shfl_sync(0xffffffffu, page_len, ((tile & 15) << 1) + j);
    }
    // V lanes: bit 0 the page, bit 1 which half of its tokens comes first, bit 2 which of two pieces comes first, bits 1 .. 4
    // the pair of pieces: any 8 lanes that store together then reach all banks.
    __device__ __forceinline__ int pair() const { return (lane >> 1) & 15; }

    __device__ __forceinline__ void load_k(const Segment &s, int tile) {
        look(s, tile);
        const unsigned char *p0 = page_of(tile, 0), *p1 = page_of(tile, 1);
        const int n0 = len_of(tile, 0), n1 = len_of(tile, 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned char *p = j < 2 ? p0 : p1;
            k[j] = p ? ld_stream16(reinterpret_cast<const uint4 *>(p) + (j & 1) * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
        }
        const unsigned char *p = lane < 16 ? p0 : p1;
        live = lane < 16 ? n0 : n1;
        mk = mv = make_uint2(0u, 0u);
        if ((lane & 15) < live) {
            mk = *reinterpret_cast<const uint2 *>(p + q4::kKMeta + (lane & 15) * 8);
            mv = *reinterpret_cast<const uint2 *>(p + q4::kVMeta + (lane & 15) * 8);
        }
    }
    __device__ __forceinline__ void load_v(const Segment &s, int tile) {
        look(s, tile);
        const unsigned char *p0 = page_of(tile, 0), *p1 = page_of(tile, 1), *p = (lane & 1) ? p1 : p0;
        const int sw = (lane >> 1) & 1, par = (lane >> 2) & 1;
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // (piece, half, token pair)
            const int pc = 2 * pair() + ((i >> 3) ^ par), tt = 4 * (((i >> 2) & 1) ^ sw) + (i & 3);
            v[i] = p ? __ldg(reinterpret_cast<const uint32_t *>(p + q4::kV) + tt * 32 + (pc & 7) * 4 + (pc >> 3)) : 0u;
        }
    }

    // (step, mid) of this lane's token: exponents, operands, and what the softmax has to know.
    __device__ __forceinline__ void put_meta(Info &info) {
        MetaScratch &M = S.meta[warp];
        const bool used = (lane & 15) < live;
        float2 a = q4::unpack_meta(mk.x), c = q4::unpack_meta(mk.y);
        int e = exponent_for(fmaxf(fabsf(a.y) + 7.5f * a.x, fabsf(c.y) + 7.5f * c.x));
        float f = pow2(-e);
        M.k[lane][0] = half2_of(a.x * f, a.y * f);
        M.k[lane][1] = half2_of(c.x * f, c.y * f);
        a = q4::unpack_meta(mv.x), c = q4::unpack_meta(mv.y);
        const int ev = exponent_for(fmaxf(fabsf(a.y) + 7.5f * a.x, fabsf(c.y) + 7.5f * c.x));
        f = pow2(-ev);
        const uint32_t x = half2_of(a.x * f, a.y * f), y = half2_of(c.x * f, c.y * f);
        uint16_t(&vm)[2][2][16] = M.v[lane >> 4];
        vm[0][0][lane & 15] = (uint16_t)x, vm[0][1][lane & 15] = (uint16_t)(x >> 16);
        vm[1][0][lane & 15] = (uint16_t)y, vm[1][1][lane & 15] = (uint16_t)(y >> 16);
        info.kf[32 * warp + lane] = pow2(e);
        info.vf[32 * warp + lane] = (float)ev;
        const uint32_t mask = __ballot_sync(0xffffffffu, used);
        const uint32_t flags = (__any_sync(0xffffffffu, e != 0) ? 1u : 0u) | (__any_sync(0xffffffffu, ev != 0) ? 2u : 0u);
        if (lane == 0) info.mask[warp] = mask, info.flags[warp] = flags;
        __syncwarp();
    }
    __device__ __forceinline__ void put_k(uint32_t dst) {
        const MetaScratch &M = S.meta[warp];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = (j >> 1) * 16 + (j & 1) * 8 + (lane >> 2), token = 32 * warp + t, i = lane & 3;
            const uint32_t m0 = M.k[t][0], m1 = M.k[t][1];
            const uint32_t s0 = __byte_perm(m0, m0, 0x1010), d0 = __byte_perm(m0, m0, 0x3232);
            const uint32_t s1 = __byte_perm(m1, m1, 0x1010), d1 = __byte_perm(m1, m1, 0x3232);
            const int odd = t & 1;  // (neighbouring tokens store different words at a time)
            const uint32_t w[4] = {odd ? k[j].y : k[j].x, odd ? k[j].x : k[j].y, odd ? k[j].w : k[j].z,
                                   odd ? k[j].z : k[j].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int c = i + 4 * ((x & 1) ^ odd);  // 16-byte column within the half of 64 elements
                const uint32_t st = x < 2 ? s0 : s1, md = x < 2 ? d0 : d1;
                sts128(dst + (x >> 1) * kHalfBytes + token * 128 + ((c ^ (token & 7)) << 4),
                       hfma2(code_pair(w[x], 0), st, md), hfma2(code_pair(w[x], 1), st, md),
                       hfma2(code_pair(w[x], 2), st, md), hfma2(code_pair(w[x], 3), st, md));
            }
        }
    }
    __device__ __forceinline__ void put_v(uint32_t dst) {
        const int pg = lane & 1, sw = (lane >> 1) & 1, par = (lane >> 2) & 1, g = pair() >> 3;
        const uint16_t(&vm)[2][16] = S.meta[warp].v[pg][g];
        const uint32_t base = dst + (warp >> 1) * kHalfBytes;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int th = hf ^ sw;
            const uint4 st = *reinterpret_cast<const uint4 *>(&vm[0][8 * th]);
            const uint4 md = *reinterpret_cast<const uint4 *>(&vm[1][8 * th]);
            const int c = ((2 * warp + pg) & 3) * 2 + th;
#pragma unroll
            for (int sl = 0; sl < 2; ++sl) {
                const int pc = 2 * pair() + (sl ^ par);
                const uint32_t *w = v + sl * 8 + hf * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = 4 * pc + e;
                    sts128(base + d * 128 + ((c ^ (d & 7)) << 4), hfma2(code_pair(w[0], e), st.x, md.x),
                           hfma2(code_pair(w[1], e), st.y, md.y), hfma2(code_pair(w[2], e), st.z, md.z),
                           hfma2(code_pair(w[3], e), st.w, md.w));
                }
            }
        }
    }

    // A tile of nodes: rows of 16 vectors of 8 elements, 16 lanes a row.
    __device__ __forceinline__ void node_k(uint32_t dst, const Segment &s, int b, int h, int j0, Info &info) {
        const int c = lane & 15;
        uint32_t flags = 0u;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int token = 32 * warp + 2 * i + (lane >> 4), node = j0 + token;
            q4::Vec8<__nv_bfloat16> w;
            w.zero();
            if (node < s.nodes) w.load(row_ptr<__nv_bfloat16>(A.k, b, node, h) + 8 * c);
            float x[8], big = 0.f;
            w.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (fabsf(x[e]) < INFINITY) big = fmaxf(big, fabsf(x[e]));
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
            const int e2 = exponent_for(big);
            const float f = pow2(-e2);
            const int col = (c & 7) ^ (token & 7);
            sts128(dst + (c >> 3) * kHalfBytes + token * 128 + (col << 4), half2_of(x[0] * f, x[4] * f),
                   half2_of(x[1] * f, x[5] * f), half2_of(x[2] * f, x[6] * f), half2_of(x[3] * f, x[7] * f));
            if (c == 0) info.kf[token] = pow2(e2);
            flags |= __any_sync(0xffffffffu, e2 != 0) ? 1u : 0u;
        }
        // (the softmax needs V's exponents with the scores, before V itself is put)
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int token = 32 * warp + 2 * i + (lane >> 4), node = j0 + token;
            q4::Vec8<__nv_bfloat16> w;
            w.zero();
            if (node < s.nodes) w.load(row_ptr<__nv_bfloat16>(A.v, b, node, h) + 8 * c);
            float x[8], big = 0.f;
            w.get(x);
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (fabsf(x[e]) < INFINITY)
                    big = fmaxf(big, fabsf(x[e]));
                else
                    bad = true;
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
            const int e2 = exponent_for(big);
            if (c == 0) info.vf[token] = (float)e2;
            flags |= __any_sync(0xffffffffu, e2 != 0) ? 2u : 0u;
            if (__any_sync(0xffffffffu, bad) && lane == 0) S.bad = 1;
        }
        if (lane == 0) info.mask[warp] = 0xffffffffu, info.flags[warp] = flags;
    }
    __device__ __forceinline__ void node_v(uint32_t dst, const Segment &s, int b, int h, int j0, const Info &info) {
        const int c = lane & 15;
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
            const int token = 32 * warp + 4 * i + 2 * (lane >> 4), node = j0 + token;  // and the next one
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

// -------------------------------------------------------- softmax threads --
// 32 scores from column `at` on, those without a bit in `mask` -inf.
__device__ __forceinline__ void load_scores(uint32_t at, uint32_t mask, float (&s)[32]) {
    tmem_ld32_nowait(at, s);
    tmem_wait_ld();
    if (mask != 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(mask >> i & 1u)) s[i] = -INFINITY;
    }
}

struct Row {
    float m, mo, l, r;  // running maxima of the scores (of the sum, of O), sum, factor of the products (> 0)
};

// Scales this thread's row of O by f (a warp at a time).
__device__ __noinline__ void scale_o(uint32_t at, float f) {
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        float x[16];
        uint32_t y[16];
        tmem_ld16_nowait(at + 16 * c, x);
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

// A tile where keys or values carry powers of two of their own, or the two maxima have parted.
__device__ __noinline__ void softmax_any(uint32_t s_at, uint32_t o_at, const Info &info, const uint32_t (&mask)[4],
                                         bool first, Row &R) {
    float top = -INFINITY, top_o = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        float s[16];
        tmem_ld16_nowait(s_at + 16 * c, s);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = mask[c >> 1] >> (16 * (c & 1) + i) & 1u ? s[i] * info.kf[16 * c + i] * R.r : -INFINITY;
            top = fmaxf(top, x);
            top_o = fmaxf(top_o, x + info.vf[16 * c + i]);
        }
    }
    float f, unused;
    float lf = 1.f;
    {
        const float before = R.m;
        raise(R.m, top, first, unused);
        lf = first ? 0.f : exp2_fast(before - R.m);
    }
    if (raise(R.mo, top_o, first, f)) scale_o(o_at, f);
    R.l = lf == 1.f ? R.l : R.l * lf;
    const float off = kTop - R.m, off_o = kTop - R.mo;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        float s[16], p[16];
        tmem_ld16_nowait(s_at + 16 * c, s);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = mask[c >> 1] >> (16 * (c & 1) + i) & 1u ? s[i] * info.kf[16 * c + i] * R.r : -INFINITY;
            R.l += exp2_fast(x + off);
            p[i] = exp2_fast(x + info.vf[16 * c + i] + off_o);
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = half2_of(p[2 * i], p[2 * i + 1]);
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(s_at + 8 * c),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    }
}

__device__ __forceinline__ void softmax_tile(uint32_t s_at, uint32_t o_at, const Info &info, const uint32_t (&mask)[4],
                                             bool first, Row &R) {
    const uint4 fl = *reinterpret_cast<const uint4 *>(info.flags);
    if (__any_sync(0xffffffffu, (fl.x | fl.y | fl.z | fl.w) != 0u || (!first && !(R.m == R.mo)))) {
        softmax_any(s_at, o_at, info, mask, first, R);
        return;
    }
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float s[32];
        load_scores(s_at + 32 * c, mask[c], s);
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, s[i]);
    }
    float f;
    if (raise(R.m, top * R.r, first, f)) {
        scale_o(o_at, f);
        R.l *= f;
    }
    if (first) R.l = 0.f;
    R.mo = R.m;
    const float off = kTop - R.m;
    const unsigned long long r2 = pk2(R.r, R.r), off2 = pk2(off, off);
    unsigned long long sum[2] = {pk2(R.l, 0.f), pk2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float s[32];
        uint32_t w[16];
        load_scores(s_at + 32 * c, mask[c], s);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 x = upk2(fma2(pk2(s[2 * i], s[2 * i + 1]), r2, off2));
            const float a = exp2_fast(x.x), b = exp2_fast(x.y);
            sum[i & 1] = add2(sum[i & 1], pk2(a, b));
            w[i] = half2_of(a, b);
        }
        tmem_st16(s_at + 16 * c, w);
    }
    const float2 l = upk2(add2(sum[0], sum[1]));
    R.l = l.x + l.y;
}

// The queries of a stream's rows (thread = row) as fp16 in shared memory (null: not written, the other stream has the same
// ones), and the factor of their products.
__device__ __forceinline__ float prepare_q(const Args &A, const Piece &P, int r, uint32_t dst, int row) {
    const float sl = A.scale * 1.4426950408889634f;
    const __nv_bfloat16 *src = nullptr;
    if (r < P.rows) src = row_ptr<__nv_bfloat16>(A.q, P.b, (P.row0 + r) / A.g, P.h * A.g + (P.row0 + r) % A.g);
    float big = 0.f;
    bool fine = true;
#pragma unroll 4
    for (int c = 0; c < 16; ++c) {
        if (!src) break;
        float x[8];
        load8<__nv_bfloat16>(src + 8 * c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[e])), fine &= fabsf(x[e]) < INFINITY;
    }
    const int e2 = min(max(14 - ((int)((__float_as_uint(big) >> 23) & 255u) - 127), -113), 126);
    const float up = sl == 0.f ? 0.f : copysignf(pow2(e2), sl);
    if (dst) {
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (src) load8<__nv_bfloat16>(src + 8 * c, x);
            sts128(dst + (c >> 3) * kHalfBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                   half2_of(x[0] * up, x[4] * up), half2_of(x[1] * up, x[5] * up), half2_of(x[2] * up, x[6] * up),
                   half2_of(x[3] * up, x[7] * up));
        }
    }
    const float f = sl == 0.f ? 1.f : fabsf(sl) * pow2(-e2);
    return fine && f < INFINITY ? fmaxf(f, FLT_MIN) : __int_as_float(0x7fc00000);
}

// Row r's bits of the nodes from j0 on.
__device__ __forceinline__ void node_mask(const Args &A, const Smem &S, int anc, int node, int j0, uint32_t (&mask)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (A.parents) {
            mask[c] = S.anc.mask[anc][node][(j0 >> 5) + c];
        } else {
            const int n = node - (j0 + 32 * c) + 1;
            mask[c] = n >= 32 ? 0xffffffffu : (n > 0 ? (1u << n) - 1u : 0u);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) k_tree_tc(const __grid_constant__ Args A) {
    extern __shared__ unsigned char smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = A.g;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.k_full[i], kLoadWarps), mbar_init(&S.k_empty[i], 1);
            mbar_init(&S.v_full[i], kLoadWarps), mbar_init(&S.v_empty[i], 1);
            mbar_init(&S.s_ready[i], 1), mbar_init(&S.p_ready[i], kSoftWarps / 2);
        }
        mbar_init(&S.q_full, kSoftWarps), mbar_init(&S.o_ready, 1), mbar_init(&S.seg_done, kSoftWarps);
        mbar_init(&S.soft, kSoftWarps);
        mbar_init_fence();
        S.dead = 0, S.bad = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(&S.tmem, 512);
    dep_wait();
    const Run run = plan_run<kTreeRowsTc, kThreads>(A, S.plan);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = S.tmem;
    Part part{0, 0, 0, 0};
    auto wait = [&](unsigned long long *bar, uint32_t parity) {
        if (*static_cast<volatile int *>(&S.dead)) return false;
        if (mbar_wait(bar, parity)) return true;
        *static_cast<volatile int *>(&S.dead) = 1;
        set_err(A.err, ICE_ERR_TIMEOUT);
        return false;
    };
    bool ok = run.n > 0;
    if (ok && warp < kSoftWarps) {
        // ---- softmax: stream g, row `row` of it
        const int st = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_at = tmem + lanes + kColS + 128 * st, o_at = tmem + lanes + kColO + 128 * st;
        uint32_t n_s = 0, n_seg = 0, tile0 = 0, n_soft = 0;
        auto soft_sync = [&] {  // a barrier of the softmax threads that gives up as every wait does
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.soft);
            ok = wait(&S.soft, n_soft++ & 1) && ok;
        };
        int anc_b = -1, anc = 0;
        Segment seg = S.plan.seg;
        for (;; next_segment<kTreeRowsTc>(A, seg)) {
            if (seg.first >= run.n) break;
            const Piece P(A, seg, run);
            if (P.n == 0) continue;  // (its tiles lie in the runs before)
            const int r = P.wide ? st * kRows + row : row;
            Row R;
            R.m = R.mo = -FLT_MAX, R.l = 0.f;
            R.r = prepare_q(A, P, r, P.wide || st == 0 ? su32(S.q[P.wide ? st : 0]) : 0u, row);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_full);
            if (A.parents && P.i0 + P.n > seg.n_page && anc_b != P.b) {
                soft_sync();  // (the last ones have been read)
                anc = find_ancestors(A.parents + (size_t)P.b * A.n_nodes, seg.nodes, S.anc, A.err, tid, 32 * kSoftWarps,
                                     soft_sync);
                anc_b = P.b;
            }
            const int node = min(P.row0 + r, P.row0 + P.rows - 1) / g;  // (rows behind the last: as the last)
            bool first = true;
            for (int i = P.wide ? 0 : st; i < P.n && ok; i += P.wide ? 1 : 2) {
                ok = wait(&S.s_ready[st], n_s++ & 1);
                if (!ok) break;
                fence_after();
                const Info &info = S.info[(tile0 + i) & (kInfos - 1)];
                uint32_t mask[4];
                if (P.i0 + i < seg.n_page) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(info.mask);
                    mask[0] = w.x, mask[1] = w.y, mask[2] = w.z, mask[3] = w.w;
                } else {
                    node_mask(A, S, anc, node, (P.i0 + i - seg.n_page) * kTile, mask);
                }
                softmax_tile(s_at, o_at, info, mask, first, R);
                first = false;
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_ready[st]);
            }
            tile0 += P.n;
            ok = ok && wait(&S.o_ready, n_seg++ & 1);
            if (!ok) break;
            fence_after();
            // ---- the row's result: O / l; less than 129 rows: the two streams' joined
            const bool whole = seg.first >= 0 && seg.end() <= run.n;
            if (!whole && seg.first >= 0) part = part_of(seg, run);
            const size_t slot = (size_t)blockIdx.x * 2 + (seg.first > 0 ? 1 : 0);
            float inv = R.l == 0.f ? 0.f : 1.f / R.l, f = 1.f;
            if (R.mo != R.m) f = exp2f(0.5f * (R.mo - R.m));
            const bool any = !first;  // (warp-uniform: this stream had a tile)
            float4 *const pass_on = reinterpret_cast<float4 *>(S.k[0]);  // [32][128]
            auto get = [&](int c, float (&x)[32]) {  // elements 32 c ..
                if (any) {
                    tmem_ld32_nowait(o_at + 32 * c, x);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = any && R.l != 0.f ? x[i] * inv * f * f : 0.f;
            };
            float w0 = 1.f, w1 = 0.f;
            if (!P.wide) {
                if (st == 1) {
                    S.join_ml[row] = make_float2(R.m, R.l);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float x[32];
                        get(c, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            pass_on[(8 * c + i) * kRows + row] =
                                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
                }
                soft_sync();
                if (st == 0) {
                    const float2 o = S.join_ml[row];
                    const float M = fmaxf(R.m, o.x);
                    w0 = R.l == 0.f ? 0.f : R.l * exp2f(R.m - M);
                    w1 = o.y == 0.f ? 0.f : o.y * exp2f(o.x - M);
                    const float L = w0 + w1;
                    R.m = M, R.l = L;
                    if (L != 0.f) w0 /= L, w1 /= L;
                }
            }
            if (P.wide || st == 0) {
                const bool out = r < P.rows;
                __nv_bfloat16 *dst = out ? row_out<__nv_bfloat16>(A.o, P.b, node, P.h * g + (P.row0 + r) % g) : nullptr;
                const int nodes0 = max(P.i0 - seg.n_page, 0) * kTile;
                const int nodes1 = min((P.i0 + P.n - seg.n_page) * kTile, seg.nodes);
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    get(c, x);
                    if (!P.wide) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 y = pass_on[(8 * c + i) * kRows + row];
                            x[4 * i] = fmaf(x[4 * i], w0, y.x * w1), x[4 * i + 1] = fmaf(x[4 * i + 1], w0, y.y * w1);
                            x[4 * i + 2] = fmaf(x[4 * i + 2], w0, y.z * w1);
                            x[4 * i + 3] = fmaf(x[4 * i + 3], w0, y.w * w1);
                        }
                    }
                    if (out && S.bad) {  // infinities and NaN of the nodes that this row sees
                        for (int j = nodes0; j < nodes1; ++j) {
                            const bool sees = A.parents ? S.anc.mask[anc][node][j >> 5] >> (j & 31) & 1u : j <= node;
                            if (!sees) continue;
                            const __nv_bfloat16 *v = row_ptr<__nv_bfloat16>(A.v, P.b, j, P.h) + 32 * c;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float y = __bfloat162float(v[i]);
                                if (!(fabsf(y) < INFINITY)) x[i] += y;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!out) break;
                        const float4 y = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        if (whole)
                            put4(dst + 32 * c + 4 * i, y);
                        else
                            A.part_o[part_at(slot, 8 * c + i, r)] = y;
                    }
                    __syncwarp();
                }
                if (out && !whole) A.part_ml[slot * kPartRows + r] = make_float2(R.m, R.l);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.seg_done);
            if (seg.end() >= run.n) break;
        }
    } else if (ok && warp < kMmaWarp) {
        // ---- unpacking
        Loader L(A, S, warp - kSoftWarps);
        uint32_t tile0 = 0, n_seg = 0;
        Segment seg = S.plan.seg;
        for (;; next_segment<kTreeRowsTc>(A, seg)) {
            if (seg.first >= run.n) break;
            const Piece P(A, seg, run);
            if (P.n == 0) continue;
            L.start(seg);
            const int pages = min(max(seg.n_page - P.i0, 0), P.n);  // tiles of pages
            if (pages > 0) L.load_k(seg, P.i0), L.load_v(seg, P.i0);
            if (n_seg > 0) ok = wait(&S.seg_done, (n_seg - 1) & 1);
            ++n_seg;
            for (int i = 0; i < P.n && ok; ++i) {
                const uint32_t at = tile0 + i, stage = at & 1, parity = (at >> 1 & 1) ^ 1;
                Info &info = S.info[at & (kInfos - 1)];
                const int j0 = (P.i0 + i - seg.n_page) * kTile;
                ok = wait(&S.k_empty[stage], parity);
                if (!ok) break;
                if (i < pages) {
                    L.put_meta(info);
                    L.put_k(su32(S.k[stage]));
                } else {
                    L.node_k(su32(S.k[stage]), seg, P.b, P.h, j0, info);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.k_full[stage]);
                ok = wait(&S.v_empty[stage], parity);
                if (!ok) break;
                if (i < pages)
                    L.put_v(su32(S.v[stage]));
                else
                    L.node_v(su32(S.v[stage]), seg, P.b, P.h, j0, info);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.v_full[stage]);
                if (i + 1 < pages) L.load_k(seg, P.i0 + i + 1), L.load_v(seg, P.i0 + i + 1);
            }
            tile0 += P.n;
            if (!ok || seg.end() >= run.n) break;
        }
    } else if (ok && lane == 0) {
        // ---- products: step x is stream x & 1's; its tile's scores, after P V of its tile before
        uint32_t tile0 = 0, n_seg = 0, n_p[2] = {0, 0};
        Segment seg = S.plan.seg;
        for (;; next_segment<kTreeRowsTc>(A, seg)) {
            if (seg.first >= run.n) break;
            const Piece P(A, seg, run);
            if (P.n == 0) continue;
            ok = wait(&S.q_full, n_seg++ & 1);
            const int steps = (P.wide ? 2 * P.n : P.n) + 2;
            for (int x = 0; x < steps && ok; ++x) {
                const int st = x & 1, i = P.wide ? x >> 1 : x, before = P.wide ? i - 1 : i - 2;
                const bool last = !P.wide || st == 1;  // the last product with a tile's operand
                if (before >= 0 && before < P.n) {
                    const uint32_t at = tile0 + before, stage = at & 1;
                    ok = wait(&S.v_full[stage], at >> 1 & 1) && wait(&S.p_ready[st], n_p[st]++ & 1);
                    if (!ok) break;
                    fence_after();
                    const uint32_t v = su32(S.v[stage]), d = tmem + kColO + 128 * st, p = tmem + kColS + 128 * st;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_ta(d, p + 8 * kk, sw128_desc(v + (kk >> 2) * kHalfBytes + (kk & 3) * 32),
                                before > (P.wide ? 0 : st) || kk > 0);
                    if (last) umma_commit(&S.v_empty[stage]);
                }
                if (i < P.n) {
                    const uint32_t at = tile0 + i, stage = at & 1;
                    ok = wait(&S.k_full[stage], at >> 1 & 1);
                    if (!ok) break;
                    fence_after();
                    const uint32_t q = su32(S.q[P.wide ? st : 0]), k = su32(S.k[stage]), d = tmem + kColS + 128 * st;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
                        umma_bf16<kIdesc>(d, sw128_desc(q + off), sw128_desc(k + off), kk > 0);
                    }
                    umma_commit(&S.s_ready[st]);
                    if (last) umma_commit(&S.k_empty[stage]);
                }
            }
            if (!ok) break;
            umma_commit(&S.o_ready);
            tile0 += P.n;
            if (seg.end() >= run.n) break;
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (tid == 0) A.parts[blockIdx.x] = part;
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_tree_tc(const Args &A, int grid, cudaStream_t s) {
    const int smem = (int)sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_tree_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_tree_tc, dim3(grid), dim3(kThreads), smem, s, A);
}

}  // namespace ice
