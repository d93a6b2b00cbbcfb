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
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float bf16_rn(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// step and mid of a group from its extremes.  T: the storage type of the
// elements; differences of bf16 values are exact in fp32 (unless their
// exponents are more than 16 apart, where the rounding is far below a code),
// those of fp32 values are taken in fp64.
template <typename T>
__device__ __forceinline__ float2 step_mid(float lo, float hi) {
    float step, mid;
    if (sizeof(T) == 2) {
        step = (hi - lo) / 15.f;
        mid = (hi + lo) * 0.5f;
    } else {
        step = (float)(((double)hi - (double)lo) / 15.0);
        mid = (float)(((double)hi + (double)lo) * 0.5);
    }
    if (!(hi - lo < INFINITY)) return make_float2(0.f, __int_as_float(0x7fc00000));
    return make_float2(bf16_rn(step), bf16_rn(mid));
}

// Code of x: rint((x - mid) / step + 7.5), ties to even, decided as if
// exactly.  The product with the reciprocal is within 2e-6 of the quotient;
// only values that near a border between two codes (1 in 50 000, and true
// ties) take the division.
template <typename T>
__device__ __forceinline__ uint32_t code_of(float x, float mid, float step, float inv) {
    const float t = fmaf(x - mid, inv, 7.5f);
    float c = rintf(t);
    if (fabsf(t - c) > 0.49999f) {
        if (sizeof(T) == 2)
            c = rintf(__fadd_rn(__fdiv_rn(x - mid, step), 7.5f));
        else
            c = (float)rint(((double)x - (double)mid) / (double)step + 7.5);
    }
    return (uint32_t)fminf(fmaxf(c, 0.f), 15.f);
}

// The word of a vector's 8 codes.
template <typename T>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float2 sm) {
    if (!(sm.x > 0.f)) return 0u;
    // below 2^-100 the reciprocal leaves fp32's normal range: scale both sides
    const bool tiny = sm.x < 7.9e-31f;
    const float up = tiny ? 1.2676506e30f : 1.f;  // 2^100
    const float step = sm.x * up, mid = sm.y * up;
    const float inv = 1.f / step;
    uint32_t w = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= code_of<T>(tiny ? x[e] * up : x[e], mid, step, inv) << (4 * e);
    return w;
}

// Quantises a row held by 8 lanes (vectors wa and wb of lane l): the words of
// both vectors, and (step, mid) of both groups in every lane.
template <typename T>
__device__ __forceinline__ void quantise_row(const float (&a)[8], const float (&b)[8], int wa, int wb, uint32_t &ca,
                                             uint32_t &cb, float2 (&sm)[2]) {
    float la = a[0], ha = a[0], lb = b[0], hb = b[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        la = min_nan(la, a[e]);
        ha = max_nan(ha, a[e]);
        lb = min_nan(lb, b[e]);
        hb = max_nan(hb, b[e]);
    }
    float lo[2] = {INFINITY, INFINITY}, hi[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if ((wa >> 3) == g) {
            lo[g] = min_nan(lo[g], la);
            hi[g] = max_nan(hi[g], ha);
        }
        if ((wb >> 3) == g) {
            lo[g] = min_nan(lo[g], lb);
            hi[g] = max_nan(hi[g], hb);
        }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], off));
            hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], off));
        }
        sm[g] = step_mid<T>(lo[g], hi[g]);
    }
    ca = codes_of<T>(a, (wa >> 3) ? sm[1] : sm[0]);
    cb = codes_of<T>(b, (wb >> 3) ? sm[1] : sm[0]);
}

// (step, mid) of a token's two groups as stored.
__device__ __forceinline__ uint2 pack_meta(const float2 (&sm)[2]) {
    const __nv_bfloat162 g0 = __floats2bfloat162_rn(sm[0].x, sm[0].y);
    const __nv_bfloat162 g1 = __floats2bfloat162_rn(sm[1].x, sm[1].y);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&g0), *reinterpret_cast<const uint32_t *>(&g1));
}
__device__ __forceinline__ float2 unpack_meta(uint32_t m) {
    return make_float2(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}

// The values that a vector's codes stand for.
__device__ __forceinline__ void values_of(uint32_t w, float2 sm, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(sm.x, (float)((w >> (4 * e)) & 15u) - 7.5f, sm.y);
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
template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[8]) {
    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(p), x);
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[8]);
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<float>(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <typename T> __device__ __forceinline__ float round_to(float x) { return x; }
template <> __device__ __forceinline__ float round_to<__nv_bfloat16>(float x) { return q4::bf16_rn(x); }

}  // namespace ice
