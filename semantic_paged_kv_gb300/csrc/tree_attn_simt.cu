// Attention of drafted tokens over 4-bit pages on the CUDA cores:
// ice_cache4_attn_tree and ice_sparse_attn_tree4 for fp32 rows.
//   O[t] = sum_j exp(scale q_t . k_j) v_j / sum_j exp(scale q_t . k_j),
// j over the unit's pages, the ancestors of node t and t itself.
//
// 64 rows and 128 tokens a tile, keys and values unpacked to fp32 in shared
// memory, 8 x 4 scores (then 8 x 4 outputs) a thread.  A warp owns 8 rows: their
// maxima and sums stay in it.  A tile's product with V is summed apart and then
// added, which keeps the rounding of long sums down.
//
// Bound by issue and latency of one CTA of 8 warps (254 registers): FMA pipe 38%, issue 51% busy.  Measured: 61 nodes of 16/1
// heads over 100,000 tokens 1.68 ms (30 TFLOP/s), three short sequences of 4/1 heads 27 us.  The same products as packed pairs of
// fp32 operations took 2.17 ms (the pairs' order costs registers).
#include <float.h>

#include "tree.cuh"

namespace ice {
namespace {

using namespace tree;

constexpr int kRows = kTreeRowsSimt, kThreads = 256;
constexpr int kKRow = kHeadDim + 4;  // padded (conflict-free 16-byte loads of 32 rows)

struct Smem {
    float k[kTile][kKRow];
    float v[kTile][kHeadDim];
    float q[kRows][kHeadDim];
    float p[kRows][kTile];
    Ancestors anc;
    int len[kTilePages];
    int bad;  // a node's value is not finite
    PlanScratch plan;
};

// One page's rows in fp32, by a warp: lane (token, group).  Slots behind `len` are zero.
__device__ __forceinline__ void unpack_page(const unsigned char *rec, int len, int slot0, Smem &S) {
    const int lane = threadIdx.x & 31, t = lane >> 1, grp = lane & 1;
    const bool live = rec && t < len;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float2 sm = make_float2(0.f, 0.f);
        if (live)
            sm = q4::unpack_meta(*reinterpret_cast<const uint32_t *>(rec + (kv ? q4::kVMeta : q4::kKMeta) + t * 8 +
                                                                      grp * 4));
        float *dst = (kv ? S.v[slot0 + t] : S.k[slot0 + t]) + grp * 64;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int w = grp * 8 + i;
            float x[8];
            q4::values_of<8>(live ? (kv ? q4::get_v(rec, t, w) : q4::get_k(rec, t, w)) : 0u, sm, x);
            reinterpret_cast<float4 *>(dst)[2 * i] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4 *>(dst)[2 * i + 1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) k_tree_simt(const __grid_constant__ Args A) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = A.g;
    if (tid == 0) S.bad = 0;
    dep_wait();
    const Run run = plan_run<kRows, kThreads>(A, S.plan);
    Part part{};
    const float sl = fminf(fmaxf(A.scale * 1.4426950408889634f, -FLT_MAX), FLT_MAX);
    int anc_b = -1;
    if (run.n > 0) {
        Segment seg = S.plan.seg;
        for (;; next_segment<kRows>(A, seg)) {
            const int i0 = (int)max(-seg.first, 0ll), i1 = (int)min((long long)seg.n, run.n - seg.first);
            if (seg.first >= run.n) break;
            if (i0 >= i1) continue;  // (its tiles lie in the runs before)
            const int b = seg.u / A.hkv, h = seg.u - b * A.hkv;
            const int row0 = seg.blk * kRows, rows = min(kRows, seg.nodes * g - row0);
            __syncthreads();  // the segment before has been read
            for (int i = tid; i < kRows * kHeadDim / 8; i += kThreads) {
                const int r = i / (kHeadDim / 8), c = i % (kHeadDim / 8) * 8;
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (r < rows) {
                    const int t = (row0 + r) / g, hh = (row0 + r) % g;
                    load8<T>(row_ptr<T>(A.q, b, t, h * g + hh) + c, x);
                }
                *reinterpret_cast<float4 *>(&S.q[r][c]) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4 *>(&S.q[r][c + 4]) = make_float4(x[4], x[5], x[6], x[7]);
            }
            if (A.parents && i1 > seg.n_page && anc_b != b) {
                find_ancestors(tid < seg.nodes ? A.parents[(size_t)b * A.n_nodes + tid] : -1, seg.nodes, S.anc, A.err, tid,
                               [] { __syncthreads(); });
                anc_b = b;
            }
            float o[8][4], m[8], l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = -FLT_MAX, l[i] = 0.f;
                o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            }
            for (int tile = i0; tile < i1; ++tile) {
                const bool nodes = tile >= seg.n_page;
                const int j0 = (tile - seg.n_page) * kTile;  // first node of the tile
                if (!nodes) {
                    const int x = tile * kTilePages + warp;
                    int len = 0;
                    const unsigned char *rec = x < pages_of(seg.cnt) ? page_at(A, seg.u, seg.cnt, x, len) : nullptr;
                    unpack_page(rec, len, warp * kPage, S);
                    if (lane == 0) S.len[warp] = len;
                } else {
                    for (int i = tid; i < kTile * kHeadDim / 8; i += kThreads) {
                        const int r = i / (kHeadDim / 8), c = i % (kHeadDim / 8) * 8;
                        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        if (j0 + r < seg.nodes) {
                            load8<T>(row_ptr<T>(A.k, b, j0 + r, h) + c, x);
                            load8<T>(row_ptr<T>(A.v, b, j0 + r, h) + c, y);
                        }
                        // infinities and NaN join the rows that see them at the end
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (!(fabsf(y[e]) < INFINITY)) S.bad = 1, y[e] = 0.f;
                        *reinterpret_cast<float4 *>(&S.k[r][c]) = make_float4(x[0], x[1], x[2], x[3]);
                        *reinterpret_cast<float4 *>(&S.k[r][c + 4]) = make_float4(x[4], x[5], x[6], x[7]);
                        *reinterpret_cast<float4 *>(&S.v[r][c]) = make_float4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<float4 *>(&S.v[r][c + 4]) = make_float4(y[4], y[5], y[6], y[7]);
                    }
                }
                __syncthreads();
                // ---- scores: rows 8 warp + i, slots lane + 32 j
                float s[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 2
                for (int d = 0; d < kHeadDim; d += 4) {
                    float4 kk[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4 *>(&S.k[lane + 32 * j][d]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 qq = *reinterpret_cast<const float4 *>(&S.q[8 * warp + i][d]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            s[i][j] = fmaf(qq.x, kk[j].x, s[i][j]);
                            s[i][j] = fmaf(qq.y, kk[j].y, s[i][j]);
                            s[i][j] = fmaf(qq.z, kk[j].z, s[i][j]);
                            s[i][j] = fmaf(qq.w, kk[j].w, s[i][j]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int node = (row0 + 8 * warp + i) / g;
                    float mx = m[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int slot = lane + 32 * j;
                        bool sees;
                        if (!nodes)
                            sees = (slot & (kPage - 1)) < S.len[slot / kPage];
                        else if (j0 + slot >= seg.nodes || node >= seg.nodes)
                            sees = false;
                        else
                            sees = A.parents ? S.anc.mask[node][(j0 + slot) >> 5] >> (slot & 31) & 1u
                                             : j0 + slot <= node;
                        s[i][j] = sees ? s[i][j] * sl : -INFINITY;
                        mx = fmaxf(mx, s[i][j]);
                    }
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const float f = exp2f(m[i] - mx);
                    m[i] = mx;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = s[i][j] == -INFINITY ? 0.f : exp2f(s[i][j] - mx);
                        sum += p;
                        S.p[8 * warp + i][lane + 32 * j] = p;
                    }
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    l[i] = fmaf(l[i], f, sum);
                    o[i][0] *= f, o[i][1] *= f, o[i][2] *= f, o[i][3] *= f;
                }
                __syncwarp();
                // ---- outputs: rows 8 warp + i, elements 4 lane ..
                float a[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i][0] = a[i][1] = a[i][2] = a[i][3] = 0.f;
#pragma unroll 2
                for (int j = 0; j < kTile; j += 4) {
                    float4 vv[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) vv[e] = *reinterpret_cast<const float4 *>(&S.v[j + e][4 * lane]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 pp = *reinterpret_cast<const float4 *>(&S.p[8 * warp + i][j]);
                        const float w[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[i][0] = fmaf(w[e], vv[e].x, a[i][0]);
                            a[i][1] = fmaf(w[e], vv[e].y, a[i][1]);
                            a[i][2] = fmaf(w[e], vv[e].z, a[i][2]);
                            a[i][3] = fmaf(w[e], vv[e].w, a[i][3]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i][0] += a[i][0], o[i][1] += a[i][1], o[i][2] += a[i][2], o[i][3] += a[i][3];
                __syncthreads();
            }
            const bool whole = seg.first >= 0 && seg.end() <= run.n;
            if (!whole && seg.first >= 0) part = part_of<kRows>(seg, run, g);
            const size_t slot = (size_t)blockIdx.x * 2 + (seg.first > 0 ? 1 : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * warp + i;
                if (r >= rows) break;
                // (all scores -inf: NaN)
                const float inv = l[i] != 0.f ? 1.f / l[i] : (whole ? __int_as_float(0x7fc00000) : 0.f);
                float4 x = make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
                if (S.bad) {
                    const int node = (row0 + r) / g, nodes1 = min((i1 - seg.n_page) * kTile, seg.nodes);
#pragma unroll 1
                    for (int j = max(i0 - seg.n_page, 0) * kTile; j < nodes1; ++j) {
                        if (!(A.parents ? S.anc.mask[node][j >> 5] >> (j & 31) & 1u : j <= node)) continue;
                        const T *v = row_ptr<T>(A.v, b, j, h) + 4 * lane;
                        auto add = [](float &to, float y) {
                            if (!(fabsf(y) < INFINITY)) to += y;
                        };
                        add(x.x, Elem<T>::load(v)), add(x.y, Elem<T>::load(v + 1));
                        add(x.z, Elem<T>::load(v + 2)), add(x.w, Elem<T>::load(v + 3));
                    }
                }
                if (whole) {
                    put4(row_out<T>(A.o, b, (row0 + r) / g, h * g + (row0 + r) % g) + 4 * lane, x);
                } else {
                    A.part_o[part_at(slot, lane, r)] = x;
                    if (lane == 0) A.part_ml[slot * kPartRows + r] = make_float2(m[i], l[i]);
                }
            }
            if (seg.end() >= run.n) break;
        }
    }
    if (tid == 0) A.parts[blockIdx.x] = part;
}

static_assert(kThreads == kMaxNodes, "a thread a node");
static_assert(sizeof(Smem) <= 227 * 1024, "one CTA an SM");

}  // namespace

cudaError_t launch_tree_simt(const Args &A, int grid, cudaStream_t s) {
    auto kern = k_tree_simt<float>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(grid), dim3(kThreads), sizeof(Smem), s, A);
}

}  // namespace ice
