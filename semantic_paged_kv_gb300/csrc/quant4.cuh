// Pages in 4 bits: the record layout and the quantiser shared by the kernels
// that write and read 4-bit records (layout and formulas in ice.h).
//
// A row (128 elements of one token's K or V) is handled by 8 lanes, each with
// two 8-element vectors A and B; vector w of a row holds elements 8 w .. 8 w +
// 7 and belongs to group w / 8.  A vector's 8 codes are one 32-bit word: a K
// word, or two 16-bit V pieces.
#pragma once

#include "common.cuh"

namespace ice {
namespace q4 {

using pair_t = unsigned long long;  // two fp32 values (common.cuh)

constexpr int kCodeBytes = kPage * kHeadDim / 2;  // K or V codes of a record
constexpr int kMetaBytes = kPage * 8;             // (step, mid) of two groups a token
constexpr int kKMeta = kCodeBytes;
constexpr int kV = kCodeBytes + kMetaBytes;
constexpr int kVMeta = kV + kCodeBytes;
constexpr int kRecord = ICE_RECORD4_BYTES;
static_assert(kVMeta + kMetaBytes == kRecord, "record layout");

// Byte offsets inside a record.
__device__ __forceinline__ int k_word(int token, int w) { return token * 64 + ((w & 3) * 4 + (w >> 2)) * 4; }
// V piece p (elements 4 p .. 4 p + 3) of a token.
__device__ __forceinline__ int v_piece(int token, int p) {
    return kV + (((token >> 1) * 8 + (p & 7)) * 4 + (p >> 3)) * 4 + (token & 1) * 2;
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Extremes of values as (min, -max), both taken by min: one exchange serves
// two values.  bf16 values stay packed, (min, -max) in one word.
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight consecutive elements of a row in their storage type.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint32_t w[4];
    using Ends = uint32_t;
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    __device__ __forceinline__ Ends ends() const {
        const uint32_t mn = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3]));
        const uint32_t mx = max2_nan(max2_nan(w[0], w[1]), max2_nan(w[2], w[3]));
        return min2_nan(__byte_perm(mn, mx, 0x5410) ^ 0x80000000u, __byte_perm(mn, mx, 0x7632) ^ 0x80000000u);
    }
    __device__ __forceinline__ static Ends none() { return 0x7F807F80u; }
    __device__ __forceinline__ static Ends join(Ends a, Ends b) { return min2_nan(a, b); }
    __device__ __forceinline__ static Ends exchange(Ends a, int off) { return __shfl_xor_sync(0xffffffffu, a, off); }
    __device__ __forceinline__ static float lo(Ends a) { return __uint_as_float(a << 16); }
    __device__ __forceinline__ static float hi(Ends a) { return -__uint_as_float(a & 0xFFFF0000u); }
};
template <> struct Vec8<float> {
    float v[8];
    struct Ends {
        float lo, neg;
    };
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
    __device__ __forceinline__ void load(const float *p) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v[e];
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x[e];
    }
    __device__ __forceinline__ Ends ends() const {
        Ends r{v[0], -v[0]};
#pragma unroll
        for (int e = 1; e < 8; ++e) r.lo = min_nan(r.lo, v[e]), r.neg = min_nan(r.neg, -v[e]);
        return r;
    }
    __device__ __forceinline__ static Ends none() { return Ends{INFINITY, INFINITY}; }
    __device__ __forceinline__ static Ends join(Ends a, Ends b) {
        return Ends{min_nan(a.lo, b.lo), min_nan(a.neg, b.neg)};
    }
    __device__ __forceinline__ static Ends exchange(Ends a, int off) {
        return Ends{__shfl_xor_sync(0xffffffffu, a.lo, off), __shfl_xor_sync(0xffffffffu, a.neg, off)};
    }
    __device__ __forceinline__ static float lo(Ends a) { return a.lo; }
    __device__ __forceinline__ static float hi(Ends a) { return -a.neg; }
};

// step and mid of a group from its extremes.  Differences of bf16 values are
// exact in fp32 (unless their exponents are more than 16 apart, where the
// rounding is far below a code); those of fp32 values are kept with their
// rounding error.  The quotient by 15 is corrected by its remainder, which
// rounds it correctly (Markstein 1990: a quotient within an ulp and a correctly
// rounded reciprocal); differences below 1e-30, whose remainder could
// underflow, are divided (fp32's in 64 bits, which hold them).  The extremes' sum can overflow where mid does not:
// mid takes their halves, which bf16 values (and fp32 ones of that size) have
// exactly.
static __device__ __noinline__ float tiny_step(float lo, float hi) {
    return (float)(((double)hi - (double)lo) / 15.0);
}
template <typename T>
__device__ __forceinline__ float2 step_mid(float lo, float hi) {
    float d, er = 0.f;
    if (sizeof(T) == 2)
        d = hi - lo;
    else
        two_sum(hi, -lo, d, er);
    const float q = d * (1.f / 15.f);
    float step = fmaf(fmaf(-15.f, q, d) + er, 1.f / 15.f, q);
    if (d < 1e-30f) step = sizeof(T) == 2 || d == 0.f ? d / 15.f : tiny_step(lo, hi);
    if (!(d < INFINITY)) return make_float2(0.f, __int_as_float(0x7fc00000));
    float mid = fmaf(hi, 0.5f, lo * 0.5f);
    if (sizeof(T) == 4 && fabsf(hi + lo) < INFINITY) mid = (hi + lo) * 0.5f;
    return make_float2(step, mid);
}

// The word of a vector's 8 codes, rint((x - mid) / step + 7.5) with ties to
// even, decided exactly without a division: with k the integer next to (x -
// mid) / step (from an approximate reciprocal; which of two neighbours it is
// does not matter), the code is k + 8 where the remainder x - mid - k step is
// positive, k + 7 where it is negative, and the even one of the two where it
// is zero.  The remainder's sign is exact: k step is (4 bits times 8), and mid
// + k step goes in as an unevaluated sum (x - mid alone would lose a tiny x).
__device__ __forceinline__ uint32_t codes_in(const float (&x)[8], float step, float mid, float inv) {
    constexpr float kBig = 12582912.f;  // 1.5 * 2^23: integers end up in the low bits
    const pair_t mid2 = pk2(mid, mid), inv2 = pk2(inv, inv), step2 = pk2(step, step), big2 = pk2(kBig, kBig);
    uint32_t w = 0u;
    auto code = [&](int e, float t, float rem) {
        const int b = __float_as_int(t);
        const bool below = __float_as_int(rem) < (b & 1);  // negative, or zero and k odd
        w |= (uint32_t)min(max(b - 0x4B400000 + 8 - (below ? 1 : 0), 0), 15) << (4 * e);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const pair_t x2 = pk2(x[2 * i], x[2 * i + 1]), t = fma2(sub2(x2, mid2), inv2, big2);
        pair_t s, er;
        two_sum2(mid2, mul2(sub2(t, big2), step2), s, er);  // (exact products: it does not matter if they are fused)
        const float2 b = upk2(t), rem = upk2(add2(sub2(sub2(x2, s), er), 0ull));  // (+ 0: no zero with a sign)
        code(2 * i, b.x, rem.x);
        code(2 * i + 1, b.y, rem.y);
    }
    return w;
}

// The same for bf16 values of an ordinary group, in three operations a pair:
// t = (x - mid) / step + 7.5 rounded to a multiple of 2^-18 (by an addition
// near 48), then to an integer, ties to even.  A true tie survives the first
// rounding: the reciprocal's error leaves (x - mid) inv within 2^-20 of the
// quotient.  Nothing else becomes a tie: with step in [2^s, 2^(s+1)) and mid at
// least 2^-9 step from every multiple of step (ordinary), x - mid - n step is
// either 0, or above 2^-10 step (|x| < 2^-10 step), or a multiple of 2^(s-17)
// (the last bits of x, mid and step), which is 2^-18 step or more.
__device__ __forceinline__ uint32_t codes_ordinary(const float (&x)[8], float mid, float inv) {
    constexpr float kBig = 12582912.f - 48.f;  // 1.5 * 2^23 - 48
    const pair_t mid2 = pk2(mid, mid), inv2 = pk2(inv, inv), snap2 = pk2(55.5f, 55.5f), big2 = pk2(kBig, kBig);
    uint32_t w = 0u - 0x4B400000u * 0x11111111u;  // the bits of 1.5 * 2^23 in every nibble
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = upk2(add2(fma2(sub2(pk2(x[2 * i], x[2 * i + 1]), mid2), inv2, snap2), big2));
        w += __float_as_uint(t.x) * (1u << (8 * i));
        w += __float_as_uint(t.y) * (16u << (8 * i));
    }
    return w;
}
// Whether codes_ordinary() holds for a group: its codes lie in 0 .. 15 without
// clamping, step's reciprocal is normal, and mid keeps its distance (above).
__device__ __forceinline__ bool ordinary(float step, float mid, float lo, float hi) {
    constexpr float kBig = 12582912.f;
    const float n = fmaf(mid, rcp_fast(step), kBig) - kBig, off = fmaf(-n, step, mid);
    return (step >= 7.9e-31f) & (hi - mid < 8.f * step) & (mid - lo <= 8.f * step) & (fabsf(mid) < 4096.f * step) &
           (fabsf(off) >= 0.001953125f * step);
}

// The same for fp32 values: t = (x - mid) / step + 7.5 within 2^-19 (x - mid
// and the sum rounded once, 2^-21 each at |x - mid| <= 8 step; a reciprocal
// within an ulp, 2^-20), so its nearest integer is the code unless t lies
// nearer than that to a border.  `far` becomes the largest distance of a t from
// its integer: codes with one above kSure are to be found the exact way (some
// 2^-15 of all values).
constexpr float kSure = 0.5f - 1.52587890625e-5f;  // 0.5 - 2^-16
__device__ __forceinline__ uint32_t codes_near(const float (&x)[8], float mid, float inv, float &far) {
    constexpr float kBig = 12582912.f;  // 1.5 * 2^23
    const pair_t mid2 = pk2(mid, mid), inv2 = pk2(inv, inv), off2 = pk2(7.5f, 7.5f), big2 = pk2(kBig, kBig);
    uint32_t w = 0u - 0x4B400000u * 0x11111111u;  // the bits of 1.5 * 2^23 in every nibble
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const pair_t t = fma2(sub2(pk2(x[2 * i], x[2 * i + 1]), mid2), inv2, off2), u = add2(t, big2);
        const float2 d = upk2(sub2(t, sub2(u, big2))), b = upk2(u);
        far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
        w += __float_as_uint(b.x) * (1u << (8 * i));
        w += __float_as_uint(b.y) * (16u << (8 * i));
    }
    return w;
}

// Codes of any group: also steps below 2^-100 (the reciprocal leaves fp32's
// normal range; both sides scaled up), mid beside fp32's largest value (mid + k
// step could overflow; scaled down, step stays above 2^-100) and extremes
// outside the codes' range by the rounding of step and mid: far outside for
// fp32 values only (mid is within half a last place of bf16 values, whose
// extremes differ by one at least).
template <typename T>
__device__ __noinline__ uint32_t codes_any(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                            float x7, float step, float mid) {
    if (!(step > 0.f)) return 0u;
    float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
    const float up = step < 7.9e-31f ? 1.2676506e30f : (fabsf(mid) > 1e38f ? 0.0009765625f : 1.f);  // 2^100, 2^-10
    if (up != 1.f) {
        step *= up, mid *= up;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= up;
    }
    if (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], mid - 9.f * step), mid + 9.f * step);
    }
    return codes_in(x, step, mid, 1.f / step);
}

// (step, mid) as stored: one word a group.
__device__ __forceinline__ float2 unpack_meta(uint32_t m) {
    return make_float2(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}

// Quantises a row held by 8 lanes (vectors wa and wb of lane l): the words of
// both vectors, and in every lane both groups' (step, mid) as stored.  Lanes 0
// .. 3 find group 0's step and mid, lanes 4 .. 7 group 1's.  live: false for
// lanes without a row, whose results mean nothing.
template <typename T>
__device__ __forceinline__ void quantise_row(const Vec8<T> &a, const Vec8<T> &b, int wa, int wb, bool live,
                                             uint32_t &ca, uint32_t &cb, uint2 &meta) {
    using V = Vec8<T>;
    const bool upper = threadIdx.x & 4;
    const typename V::Ends ea = a.ends(), eb = b.ends();
    const typename V::Ends e0 = V::join((wa >> 3) == 0 ? ea : V::none(), (wb >> 3) == 0 ? eb : V::none());
    const typename V::Ends e1 = V::join((wa >> 3) == 1 ? ea : V::none(), (wb >> 3) == 1 ? eb : V::none());
    typename V::Ends e = V::join(upper ? e1 : e0, V::exchange(upper ? e0 : e1, 4));
    e = V::join(e, V::exchange(e, 1));
    e = V::join(e, V::exchange(e, 2));
    const float lo = V::lo(e), hi = V::hi(e);
    const float2 exact = step_mid<T>(lo, hi);
    const __nv_bfloat162 held = __floats2bfloat162_rn(exact.x, exact.y);
    const uint32_t own = *reinterpret_cast<const uint32_t *>(&held), other = __shfl_xor_sync(0xffffffffu, own, 4);
    const float2 sm = unpack_meta(own);
    meta = upper ? make_uint2(other, own) : make_uint2(own, other);
    const float2 ga = unpack_meta((wa >> 3) ? meta.y : meta.x), gb = unpack_meta((wb >> 3) ? meta.y : meta.x);
    float x[8], y[8];
    a.get(x);
    b.get(y);
    if (sizeof(T) == 2 && __all_sync(0xffffffffu, ordinary(sm.x, sm.y, lo, hi) | !live)) {
        ca = codes_ordinary(x, ga.y, rcp_fast(ga.x));
        cb = codes_ordinary(y, gb.y, rcp_fast(gb.x));
        return;
    }
    if (sizeof(T) == 4) {
        float far = 0.f;
        ca = codes_near(x, ga.y, rcp_fast(ga.x), far);
        cb = codes_near(y, gb.y, rcp_fast(gb.x), far);
        const bool fits = (sm.x >= 7.9e-31f) & (hi - sm.y <= 8.f * sm.x) & (sm.y - lo <= 8.f * sm.x);
        if (__all_sync(0xffffffffu, (fits & (far < kSure)) | !live)) return;
    }
    ca = codes_any<T>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], ga.x, ga.y);
    cb = codes_any<T>(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], gb.x, gb.y);
}

// The values that the first n codes of a word stand for: mid + step (code -
// 7.5), one rounding.  A code at bit 7 of 2^16 adds its value.
template <int n> __device__ __forceinline__ void values_of(uint32_t w, float2 sm, float (&x)[n]) {
    const pair_t step = pk2(sm.x, sm.x), mid = pk2(sm.y, sm.y), off = pk2(65543.5f, 65543.5f);
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const uint32_t a = i == 0 ? w << 7 : w >> (i == 0 ? 0 : 8 * i - 7), b = i == 0 ? w << 3 : w >> (i == 0 ? 0 : 8 * i - 3);
        const pair_t c = sub2(pk2(__uint_as_float((a & 0x780u) | 0x47800000u),
                                  __uint_as_float((b & 0x780u) | 0x47800000u)), off);
        const float2 y = upk2(fma2(step, c, mid));
        x[2 * i] = y.x, x[2 * i + 1] = y.y;
    }
}

// Writes a row's codes and (step, mid) into a record (shared or global
// memory): lane l of the row's 8.
__device__ __forceinline__ void put_k(unsigned char *rec, int token, int wa, int wb, uint32_t ca, uint32_t cb) {
    *reinterpret_cast<uint32_t *>(rec + k_word(token, wa)) = ca;
    *reinterpret_cast<uint32_t *>(rec + k_word(token, wb)) = cb;
}
__device__ __forceinline__ void put_v(unsigned char *rec, int token, int wa, int wb, uint32_t ca, uint32_t cb) {
    *reinterpret_cast<uint16_t *>(rec + v_piece(token, 2 * wa)) = (uint16_t)ca;
    *reinterpret_cast<uint16_t *>(rec + v_piece(token, 2 * wa + 1)) = (uint16_t)(ca >> 16);
    *reinterpret_cast<uint16_t *>(rec + v_piece(token, 2 * wb)) = (uint16_t)cb;
    *reinterpret_cast<uint16_t *>(rec + v_piece(token, 2 * wb + 1)) = (uint16_t)(cb >> 16);
}
__device__ __forceinline__ uint32_t get_k(const unsigned char *rec, int token, int w) {
    return *reinterpret_cast<const uint32_t *>(rec + k_word(token, w));
}
__device__ __forceinline__ uint32_t get_v(const unsigned char *rec, int token, int w) {
    return (uint32_t)*reinterpret_cast<const uint16_t *>(rec + v_piece(token, 2 * w)) |
           ((uint32_t)*reinterpret_cast<const uint16_t *>(rec + v_piece(token, 2 * w + 1)) << 16);
}

}  // namespace q4

// ------------------------------------------------ rows in 8-element vectors --
template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    q4::Vec8<T> v;
    v.load(p);
    v.get(x);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    q4::Vec8<T> v;
    v.set(x);
    v.store(p);
}

}  // namespace ice
