// Verification of drafted tokens: ice_tree_verify.
//
// At node i of a walk from node 0, with p = target[i] and q = draft[i], its
// children are tried in order.  After refusals the distribution to draw from is
//   rest = max(p - beta q, 0), mass = sum rest,
// because refusing a token once more turns rest / mass into max(rest / mass -
// q, 0), which is max(p - (beta + mass) q, 0) / mass: one number a refusal, and
// one pass over two rows to find the next mass.  Everything else is the few
// probabilities of the drafted tokens themselves, gathered ahead of the walk.
//
// One cluster of 8 CTAs a sequence: each takes an eighth of a row; all of them
// make the same walk from the same numbers, so only sums cross the cluster.
// Sums are kept as unevaluated pairs of fp32 values (48 bits; fp64 runs at 2
// operations a clock and SM here, and a row of 128000 would take 8 us a pass):
// a decision differs from exact arithmetic only where it lies within about
// 1e-12 of its border.  The order of additions is fixed, so a call always gives
// the same answer.
//
// Where no child of a node was refused its weights are p alone, and q's row is not read.
//
// Bound by latencies: the gather (parents, tokens, probabilities: three loads one after another), then about 2.5 us a refusal
// (its pass over two rows, a cluster barrier, 64 sums read across it) and the draw.  Measured, by the refusals of four draws: a
// tree of 26 nodes over 128,000 fp32 probabilities 14.1 to 26.6 us, 64 trees of up to 61 nodes in bf16 41 to 52 us (greedy 18 to
// 24 us, a pass a node of the path, and 17 to 22).  Two CTAs an SM with four vectors a lane ahead; three with two ahead take 14.2
// to 27.8 and 37 to 50 us, four with two ahead (spills) 14.2 to 32.1 and 35 to 43.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace ice {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8, kThreads = 256, kWarps = kThreads / 32, kPieces = kCluster * kWarps;
constexpr int kMaxNodes = ICE_VERIFY_NODES;

struct VerifyArgs {
    const void *target, *draft;
    long long t_batch, t_node, d_batch, d_node;
    int vocab, n_nodes, batch;
    const int32_t *parents, *counts, *tokens;
    const float *uniform;
    int32_t *path, *n_path, *next, *err;
};

// A sum as hi + lo.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
    float s, e;
    two_sum(a.hi, b.hi, s, e);
    e += a.lo + b.lo;
    Two r;
    r.hi = s + e;
    r.lo = e - (r.hi - s);
    return r;
}
__device__ __forceinline__ double value(Two a) { return (double)a.hi + (double)a.lo; }

// What a probability counts as: NaN and negative ones as 0.
__device__ __forceinline__ float counted(float x) { return fmaxf(x, 0.f); }

// max(p - beta q, 0) with beta = (bh, bl) > 0.  (A p of NaN or below 0 fails the last comparison, and so does an infinite q.)
__device__ __forceinline__ Two rest_of(float p, float q, float bh, float bl) {
    q = counted(q);
    const float hi = bh * q, lo = fmaf(bh, q, -hi);
    float s, e;
    two_sum(p, -hi, s, e);
    e -= fmaf(bl, q, lo);
    Two r;
    r.hi = s + e;
    r.lo = e - (r.hi - s);
    return r.hi > 0.f ? r : Two{0.f, 0.f};
}

// Sums of two rows of weights at once, in packed pairs of fp32 operations (common.cuh).
struct Sums {
    unsigned long long hi, lo;
    __device__ __forceinline__ void add(unsigned long long s, unsigned long long e) {
        unsigned long long t, r;
        two_sum2(hi, s, t, r);
        hi = t;
        lo = add2(lo, add2(r, e));
    }
    __device__ __forceinline__ Two total() const {
        const float2 h = upk2(hi), l = upk2(lo);
        Two a, b;
        a.hi = h.x + l.x, a.lo = l.x - (a.hi - h.x);
        b.hi = h.y + l.y, b.lo = l.y - (b.hi - h.y);
        return ice::add(a, b);
    }
};
// max(p - beta q, 0) of two elements, as s + e.
__device__ __forceinline__ void rests_of(float2 p, float2 q, float bh, float bl, unsigned long long &s,
                                         unsigned long long &e) {
    const unsigned long long q2 = pk2(counted(q.x), counted(q.y)), b2 = pk2(bh, bh), less = mul2(pk2(-bh, -bh), q2);
    two_sum2(pk2(p.x, p.y), less, s, e);
    e = sub2(e, fma2(pk2(bl, bl), q2, fma2(b2, q2, less)));
    float2 x = upk2(s), y = upk2(e);
    if (!(x.x + y.x > 0.f)) x.x = y.x = 0.f;
    if (!(x.y + y.y > 0.f)) x.y = y.y = 0.f;
    s = pk2(x.x, x.y), e = pk2(y.x, y.y);
}

// What the CTAs do next: nothing more, sum the weights of a node, find its likeliest token.
enum { kDone = 0, kSum = 1, kLargest = 2 };
struct Command {
    int op, node;
    float bh, bl;  // beta
    int plain;     // the weights are p itself
};

struct Smem {
    int32_t parent[kMaxNodes], token[kMaxNodes];
    float px[kMaxNodes], qx[kMaxNodes], u[kMaxNodes];  // p and q of a node's token at its parent
    uint8_t at_once[kMaxNodes];                        // whether it is accepted as its parent's first child
    int32_t out[kMaxNodes];                            // tokens left out at this node (no draft probabilities)
    int n_out, n_path;
    Command cmd;
    // of this CTA's warps' pieces, in two passes in turn (read by the whole cluster): sums; the largest element
    Two part[2][kWarps];
    float best[2][kWarps];
    int best_at[2][kWarps];
    // the draw: a piece, the sum before it and the sum to pass
    int piece, first, last;
    double start, want, warp_sum[kWarps];
};

__device__ __forceinline__ void join_best(float &best, int &at, float y, int k) {
    if (k >= 0 && (at < 0 || better(y, k, best, at))) best = y, at = k;
}

template <typename T> __global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 2)
    k_tree_verify(const __grid_constant__ VerifyArgs A) {
    __shared__ Smem S;
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster.block_rank(), b = blockIdx.x / kCluster, n_nodes = A.n_nodes;
    const T *target = static_cast<const T *>(A.target) + (long long)b * A.t_batch;
    const T *draft = A.draft ? static_cast<const T *>(A.draft) + (long long)b * A.d_batch : nullptr;
    int32_t *path = A.path + (size_t)b * n_nodes;
    dep_wait();
    const int nodes = A.counts ? min(max(A.counts[b], 0), n_nodes) : n_nodes;
    const bool greedy = !A.uniform;
    if (nodes == 0) {  // (the whole cluster)
        if (rank == 0) {
            for (int t = tid; t < n_nodes; t += kThreads) path[t] = -1;
            if (tid == 0) A.n_path[b] = 0, A.next[b] = -1;
        }
        return;
    }
    for (int t = tid; t < nodes; t += kThreads) {
        int up = t == 0 ? -1 : (A.parents ? A.parents[(size_t)b * n_nodes + t] : t - 1);
        if (up >= t || up < -1) {
            set_err(A.err, ICE_ERR_INVALID_ARG);
            up = -1;
        }
        int x = -1;
        float px = 0.f, qx = 0.f;
        if (up >= 0) {
            x = A.tokens[(size_t)b * n_nodes + t];
            if (x < 0 || x >= A.vocab) {
                set_err(A.err, ICE_ERR_CAPACITY);
                x = -1;
            } else if (!greedy) {
                px = counted(Elem<T>::load(target + up * A.t_node + x));
                if (draft) qx = counted(Elem<T>::load(draft + up * A.d_node + x));
            }
        }
        const float u = greedy ? 0.f : A.uniform[(size_t)b * n_nodes + t];
        S.parent[t] = up, S.token[t] = x, S.px[t] = px, S.qx[t] = qx, S.u[t] = u;
        S.at_once[t] = draft ? (double)u * (double)qx < (double)px : u < px;  // (48 bits: exact)
    }
    if (tid == 0) S.n_out = 0;
    __syncthreads();

    // The rows of a node: `head` elements before p's first whole 16-byte vector, the whole vectors, the rest.  q's row is
    // read in vectors too where it starts at the same place of one.
    constexpr int kVec = 16 / (int)sizeof(T);
    struct Rows {
        const T *p, *q;
        int head, vecs, per;  // vectors: all, of a warp's piece
        bool same;
    };
    auto rows_of = [&](int node) {
        Rows r;
        r.p = target + node * A.t_node, r.q = draft ? draft + node * A.d_node : nullptr;
        const int at = (int)(reinterpret_cast<uintptr_t>(r.p) / sizeof(T) % kVec);
        r.head = min((kVec - at) % kVec, A.vocab);
        r.vecs = (A.vocab - r.head) / kVec;
        r.same = r.q && (int)(reinterpret_cast<uintptr_t>(r.q) / sizeof(T) % kVec) == at;
        r.per = (r.vecs + kPieces - 1) / kPieces;
        return r;
    };
    // First element of piece g (warp g % kWarps of CTA g / kWarps): the head goes to the first, the rest to the last.
    auto piece = [&](const Rows &r, int g) {
        return g == 0 ? 0 : (g == kPieces ? A.vocab : r.head + min(g * r.per, r.vecs) * kVec);
    };
    // (beta is at least 1 where a child was refused; without one q's row, which may hold anything at a leaf, is not read)
    auto takes_q = [&](const Command &c) { return draft && !c.plain && c.bh > 0.f; };
    auto weight_of = [&](const Command &c, int i, float p, float q) {
        if (takes_q(c)) return rest_of(p, q, c.bh, c.bl);
        Two r{p > 0.f ? p : 0.f, 0.f};
        if (!c.plain)
            for (int j = 0; j < S.n_out; ++j)
                if (S.out[j] == i) r.hi = 0.f;
        return r;
    };
    auto weight = [&](const Command &c, const Rows &r, int i) {
        return weight_of(c, i, Elem<T>::load(r.p + i), takes_q(c) ? Elem<T>::load(r.q + i) : 0.f);
    };
    // Calls use(v, raw p, raw q) for the vectors of this lane in piece g, several of them on their way at a time.
    constexpr int kAhead = 4;
    auto for_vectors = [&](const Rows &r, bool with_q, int g, auto use) {
        const int v1 = min((g + 1) * r.per, r.vecs);
        for (int v = g * r.per + lane; v < v1; v += 32 * kAhead) {
            uint4 p[kAhead], q[kAhead];
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
                const int i = r.head + min(v + 32 * h, v1 - 1) * kVec;
                p[h] = __ldg(reinterpret_cast<const uint4 *>(r.p + i));
                if (with_q && r.same) {
                    q[h] = __ldg(reinterpret_cast<const uint4 *>(r.q + i));
                } else if (with_q) {
                    union {
                        T x[kVec];
                        uint4 v;
                    } y;
#pragma unroll
                    for (int e = 0; e < kVec; ++e) y.x[e] = r.q[i + e];
                    q[h] = y.v;
                }
            }
#pragma unroll
            for (int h = 0; h < kAhead; ++h)
                if (v + 32 * h < v1) use(r.head + (v + 32 * h) * kVec, p[h], q[h]);
        }
    };

    // ---- the walk, by warp 0 of every CTA: children up to `tried` have been tried
    int node = 0, tried = 0, n_path = 1, likeliest = -1, pass = 0;
    double beta = 0., mass = 1., sum = 0.;
    bool fresh = true;           // no child of `node` has been refused
    Two two[2] = {};             // sums of pieces 2 lane and 2 lane + 1
    bool summed = false, searched = false;  // `sum` and the parts are those of the next command's weights
    Command cmd{kDone, 0, 0.f, 0.f, 0};
    if (tid == 0 && rank == 0) path[0] = 0;
    for (;;) {
        if (warp == 0) {
            cmd.op = greedy && !searched ? kLargest : -1;
            while (cmd.op < 0) {
                int c = -1;  // the next child
                for (int at = (tried + 1) & ~31; at < nodes && c < 0; at += 32) {
                    const int t = at + lane;
                    const unsigned hit = __ballot_sync(0xffffffffu, t < nodes && t > tried && S.parent[t] == node);
                    if (hit) c = at + __ffs(hit) - 1;
                }
                if (c < 0) {  // none left: the draw, from weights that have been summed
                    cmd.op = kDone;
                    if (!greedy && !summed) cmd.op = kSum;
                    if (!greedy && summed && !(sum > 0.) && !cmd.plain) cmd.op = kSum, cmd.plain = 1;
                    break;
                }
                tried = c;
                const int x = S.token[c];
                if (x < 0) continue;
                bool take;
                if (greedy) {
                    take = x == likeliest;
                } else if (draft) {
                    if (fresh) {
                        take = S.at_once[c];
                    } else {
                        const double px = S.px[c], qx = S.qx[c];
                        take = (double)S.u[c] * qx * mass < px - beta * qx;
                    }
                    if (!take && mass > 0.) beta += mass, cmd.op = kSum;
                } else {
                    bool gone = false;
                    for (int i = lane; i < S.n_out; i += 32) gone |= S.out[i] == x;
                    const float px = __any_sync(0xffffffffu, gone) ? 0.f : S.px[c];
                    take = fresh ? S.at_once[c] : (double)S.u[c] * mass < (double)px;
                    if (!take && px > 0.f) {
                        mass = fmax(mass - (double)px, 0.);
                        summed = false;
                        __syncwarp();
                        if (lane == 0) S.out[S.n_out++] = x;
                        __syncwarp();
                    }
                }
                fresh = false;
                if (take) {
                    fresh = true;
                    if (rank == 0 && lane == 0) path[n_path] = c;
                    ++n_path;
                    node = tried = c, beta = 0., mass = 1., summed = false;
                    __syncwarp();
                    if (lane == 0) S.n_out = 0;
                    __syncwarp();
                    if (greedy) cmd.op = kLargest;
                }
            }
            cmd.node = node;
            cmd.bh = (float)beta, cmd.bl = (float)(beta - (double)cmd.bh);
            if (lane == 0) S.cmd = cmd;
        }
        __syncthreads();
        cmd = S.cmd;
        if (cmd.op == kDone) break;
        const Rows r = rows_of(cmd.node);
        const int g = rank * kWarps + warp;
        const bool with_q = takes_q(cmd);
        // (elements outside the whole vectors: one a lane, behind the others)
        const int edge = g == 0 && lane < r.head ? lane
                         : g == kPieces - 1 && r.head + r.vecs * kVec + lane < A.vocab && lane < kVec
                             ? r.head + r.vecs * kVec + lane
                             : -1;
        if (cmd.op == kSum) {
            Sums s[2] = {{0ull, 0ull}, {0ull, 0ull}};
            for_vectors(r, with_q, g, [&](int i, const uint4 &pv, const uint4 &qv) {
                float p[kVec], q[kVec];
                Elem<T>::unpack(pv, p);
                if (with_q) Elem<T>::unpack(qv, q);
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    unsigned long long w, d = 0ull;
                    if (with_q)
                        rests_of(make_float2(p[e], p[e + 1]), make_float2(q[e], q[e + 1]), cmd.bh, cmd.bl, w, d);
                    else
                        w = pk2(weight_of(cmd, i + e, p[e], 0.f).hi, weight_of(cmd, i + e + 1, p[e + 1], 0.f).hi);
                    s[e >> 1 & 1].add(w, d);
                }
            });
            Two t = add(s[0].total(), s[1].total());
            if (edge >= 0) t = add(t, weight(cmd, r, edge));
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                t = add(t, Two{__shfl_xor_sync(0xffffffffu, t.hi, off), __shfl_xor_sync(0xffffffffu, t.lo, off)});
            if (lane == 0) S.part[pass & 1][warp] = t;
        } else {
            float best = -INFINITY;
            int at = -1;
            for_vectors(r, false, g, [&](int i, const uint4 &pv, const uint4 &) {
                float p[kVec];
                Elem<T>::unpack(pv, p);
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (p[e] > 0.f) join_best(best, at, p[e], i + e);  // (counted(p) = 0 is no probability)
            });
            if (edge >= 0) {
                const float x = Elem<T>::load(r.p + edge);
                if (x > 0.f) join_best(best, at, x, edge);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                const float y = __shfl_xor_sync(0xffffffffu, best, off);
                join_best(best, at, y, __shfl_xor_sync(0xffffffffu, at, off));
            }
            if (lane == 0) S.best[pass & 1][warp] = best, S.best_at[pass & 1][warp] = at;
        }
        cluster.sync();
        if (warp == 0) {  // pieces 2 lane and 2 lane + 1
            static_assert(kPieces == 64 && kWarps % 2 == 0, "two pieces a lane");
            const Smem *o = cluster.map_shared_rank(&S, 2 * lane / kWarps);
            const int w = 2 * lane % kWarps;
            if (cmd.op == kSum) {
                two[0] = o->part[pass & 1][w], two[1] = o->part[pass & 1][w + 1];
                Two t = add(two[0], two[1]);
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1)
                    t = add(t, Two{__shfl_xor_sync(0xffffffffu, t.hi, off), __shfl_xor_sync(0xffffffffu, t.lo, off)});
                // (the lanes' orders of addition differ: the first one's)
                sum = value(Two{__shfl_sync(0xffffffffu, t.hi, 0), __shfl_sync(0xffffffffu, t.lo, 0)});
                summed = true;
                if (draft && !cmd.plain) mass = sum;
            } else {
                float best = o->best[pass & 1][w];
                int at = o->best_at[pass & 1][w];
                join_best(best, at, o->best[pass & 1][w + 1], o->best_at[pass & 1][w + 1]);
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) {
                    const float y = __shfl_xor_sync(0xffffffffu, best, off);
                    join_best(best, at, y, __shfl_xor_sync(0xffffffffu, at, off));
                }
                likeliest = at;
                searched = true;
            }
        }
        ++pass;
    }
    cluster.barrier_arrive();  // (the others' sums have been read; they may leave while this CTA draws)
    // ---- the draw: the piece, the thread's stretch of it and the element where the running sum passes u sum (behind
    // roundings, or with u = 1: the last element of any weight)
    if (warp == 0) {
        int chosen = -1;
        if (!greedy && sum > 0.) {
            const double want = (double)S.u[0] * sum, a = value(two[0]), w = a + value(two[1]);
            double s = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, s, off);
                if (lane >= off) s += y;
            }
            const unsigned some = __ballot_sync(0xffffffffu, w > 0.), hit = __ballot_sync(0xffffffffu, w > 0. && s > want);
            const int k = hit ? __ffs(hit) - 1 : 31 - __clz(some);
            const double from = s - w;
            const bool second = !(a > 0. && from + a > want) && value(two[1]) > 0.;
            chosen = __shfl_sync(0xffffffffu, 2 * lane + (second ? 1 : 0), k);
            const double start = __shfl_sync(0xffffffffu, second ? from + a : from, k);
            if (lane == 0) S.start = start, S.want = want;
        } else if (!greedy && rank == 0 && lane == 0) {
            A.next[b] = -1;
            set_err(A.err, ICE_ERR_INVALID_ARG);
        }
        if (lane == 0) S.piece = chosen, S.first = kThreads, S.last = -1, S.n_path = n_path;
    }
    __syncthreads();
    if (S.piece >= 0 && S.piece / kWarps == rank) {
        const Rows r = rows_of(cmd.node);
        const int i0 = piece(r, S.piece), i1 = piece(r, S.piece + 1), stretch = (i1 - i0 + kThreads - 1) / kThreads;
        const int j0 = min(i0 + tid * stretch, i1), j1 = min(j0 + stretch, i1);
        Two t{0.f, 0.f};
#pragma unroll 8
        for (int j = j0; j < j1; ++j) t = add(t, weight(cmd, r, j));
        const double w = value(t);
        double s = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        if (lane == 31) S.warp_sum[warp] = s;
        __syncthreads();
        double from = S.start;
        for (int k = 0; k < warp; ++k) from += S.warp_sum[k];
        from += s - w;
        const unsigned some = __ballot_sync(0xffffffffu, w > 0.);
        const unsigned hit = __ballot_sync(0xffffffffu, w > 0. && from + w > S.want);
        if (lane == 0 && hit) atomicMin(&S.first, 32 * warp + __ffs(hit) - 1);
        if (lane == 0 && some) atomicMax(&S.last, 32 * warp + 31 - __clz(some));
        __syncthreads();
        if (tid == (S.first < kThreads ? S.first : S.last)) {
            int x = -1;
            for (int j = j0; j < j1; ++j) {
                const double y = value(weight(cmd, r, j));
                if (!(y > 0.)) continue;
                x = j;
                from += y;
                if (from > S.want) break;
            }
            A.next[b] = x;
        }
    }
    // behind the path: -1
    if (rank == 0) {
        n_path = S.n_path;
        for (int t = n_path + tid; t < n_nodes; t += kThreads) path[t] = -1;
        if (tid == 0) {
            A.n_path[b] = n_path;
            if (greedy) {
                A.next[b] = likeliest;
                if (likeliest < 0) set_err(A.err, ICE_ERR_INVALID_ARG);
            }
        }
    }
    cluster.barrier_wait();  // (the others may still read this CTA's sums)
}

}  // namespace

cudaError_t launch_tree_verify(int batch, int vocab, int dtype, const ice_tree &t, const ice_probs &target,
                               const ice_probs *draft, const int32_t *tokens, const float *uniform, int32_t *path,
                               int32_t *n_path, int32_t *next, int32_t *err, cudaStream_t s) {
    VerifyArgs A{};
    A.target = target.data, A.t_batch = target.batch, A.t_node = target.node;
    if (draft) A.draft = draft->data, A.d_batch = draft->batch, A.d_node = draft->node;
    A.vocab = vocab, A.n_nodes = t.n_nodes, A.batch = batch;
    A.parents = t.parents, A.counts = t.counts, A.tokens = tokens, A.uniform = uniform;
    A.path = path, A.n_path = n_path, A.next = next, A.err = err;
    auto kern = dtype == ICE_BF16 ? k_tree_verify<__nv_bfloat16> : k_tree_verify<float>;
    return launch_dependent(kern, dim3(batch * kCluster), dim3(kThreads), 0, s, A);
}

}  // namespace ice
