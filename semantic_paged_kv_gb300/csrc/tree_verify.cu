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
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace ice {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8, kThreads = 512, kWarps = kThreads / 32;
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

// max(p - beta q, 0) with beta = (bh, bl); NaN counts as 0.
__device__ __forceinline__ Two rest_of(float p, float q, float bh, float bl) {
    const float hi = bh * q, lo = fmaf(bh, q, -hi);
    float s, e;
    two_sum(p, -hi, s, e);
    e -= fmaf(bl, q, lo);
    Two r;
    r.hi = s + e;
    r.lo = e - (r.hi - s);
    return r.hi > 0.f ? r : Two{0.f, 0.f};
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
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
    int32_t out[kMaxNodes];                            // tokens left out at this node (no draft probabilities)
    int n_out, n_path;
    Command cmd;
    Two part[kWarps];  // sums of the warps' pieces
    float part_best[kWarps];
    int part_at[kWarps];
    // of this CTA, in two passes in turn (read by the whole cluster)
    Two total[2];
    float best[2];
    int best_at[2];
};

__device__ __forceinline__ void join_best(float &best, int &at, float y, int k) {
    if (k >= 0 && (at < 0 || better(y, k, best, at))) best = y, at = k;
}

template <typename T> __global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
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
                px = Elem<T>::load(target + up * A.t_node + x);
                if (draft) qx = Elem<T>::load(draft + up * A.d_node + x);
            }
        }
        S.parent[t] = up, S.token[t] = x, S.px[t] = px, S.qx[t] = qx;
        S.u[t] = greedy ? 0.f : A.uniform[(size_t)b * n_nodes + t];
    }
    if (tid == 0) S.n_out = 0;
    __syncthreads();

    // A warp's piece of a row: per elements from i0 on.
    const int per = (A.vocab + kCluster * kWarps - 1) / (kCluster * kWarps);
    auto piece = [&](int w) { return min((rank * kWarps + w) * per, A.vocab); };
    auto weight = [&](const Command &c, int i) {
        const float x = Elem<T>::load(target + c.node * A.t_node + i);
        if (draft && !c.plain) return rest_of(x, Elem<T>::load(draft + c.node * A.d_node + i), c.bh, c.bl);
        Two r{x > 0.f ? x : 0.f, 0.f};
        if (!c.plain)
            for (int j = 0; j < S.n_out; ++j)
                if (S.out[j] == i) r.hi = 0.f;
        return r;
    };

    // ---- the walk, by warp 0 of every CTA: children up to `tried` have been tried
    int node = 0, tried = 0, n_path = 1, likeliest = -1, pass = 0;
    double beta = 0., mass = 1., sum = 0.;
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
                    const double px = S.px[c], qx = S.qx[c];
                    take = (double)S.u[c] * qx * mass < px - beta * qx;
                    if (!take && mass > 0.) beta += mass, cmd.op = kSum;
                } else {
                    bool gone = false;
                    for (int i = lane; i < S.n_out; i += 32) gone |= S.out[i] == x;
                    const float px = __any_sync(0xffffffffu, gone) ? 0.f : S.px[c];
                    take = (double)S.u[c] * mass < (double)px;
                    if (!take && px > 0.f) {
                        mass = fmax(mass - (double)px, 0.);
                        summed = false;
                        __syncwarp();
                        if (lane == 0) S.out[S.n_out++] = x;
                        __syncwarp();
                    }
                }
                if (take) {
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
        const int i0 = piece(warp), i1 = piece(warp + 1);
        if (cmd.op == kSum) {
            Two s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = Two{0.f, 0.f};
            for (int i = i0 + lane; i < i1; i += 128)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + 32 * k < i1) s[k] = add(s[k], weight(cmd, i + 32 * k));
            Two t = add(add(s[0], s[1]), add(s[2], s[3]));
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                t = add(t, Two{__shfl_xor_sync(0xffffffffu, t.hi, off), __shfl_xor_sync(0xffffffffu, t.lo, off)});
            if (lane == 0) S.part[warp] = t;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kWarps; ++w) t = add(t, S.part[w]);
                S.total[pass & 1] = t;
            }
        } else {
            const T *p = target + cmd.node * A.t_node;
            float best = -INFINITY;
            int at = -1;
            for (int i = i0 + lane; i < i1; i += 32) {
                const float x = Elem<T>::load(p + i);
                if (x == x) join_best(best, at, x, i);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                const float y = __shfl_xor_sync(0xffffffffu, best, off);
                join_best(best, at, y, __shfl_xor_sync(0xffffffffu, at, off));
            }
            if (lane == 0) S.part_best[warp] = best, S.part_at[warp] = at;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kWarps; ++w) join_best(best, at, S.part_best[w], S.part_at[w]);
                S.best[pass & 1] = best, S.best_at[pass & 1] = at;
            }
        }
        cluster.sync();
        if (warp == 0) {
            const Smem *o = cluster.map_shared_rank(&S, lane & (kCluster - 1));
            if (cmd.op == kSum) {
                const Two t = o->total[pass & 1];
                sum = 0.;
                for (int r = 0; r < kCluster; ++r)
                    sum += value(Two{__shfl_sync(0xffffffffu, t.hi, r), __shfl_sync(0xffffffffu, t.lo, r)});
                summed = true;
                if (draft && !cmd.plain) mass = sum;
            } else {
                float best = o->best[pass & 1];
                int at = o->best_at[pass & 1];
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1) {
                    const float y = __shfl_xor_sync(0xffffffffu, best, off);
                    join_best(best, at, y, __shfl_xor_sync(0xffffffffu, at, off));
                }
                likeliest = at;
                searched = true;
            }
        }
        ++pass;
    }
    // ---- the draw: the CTA, the warp's piece, the lane's stretch and the element where the running sum passes u sum
    // (behind roundings, or with u = 1: the last element of any weight)
    if (warp == 0 && !greedy) {
        if (!(sum > 0.)) {
            if (rank == 0 && lane == 0) {
                A.next[b] = -1;
                set_err(A.err, ICE_ERR_INVALID_ARG);
            }
        } else {
            const double want = (double)S.u[0] * sum;
            double start = 0.;
            bool passed = false;
            // the first of n values (lane's w; lanes in order) whose running sum from `start` on is beyond `want`; `start`
            // becomes the sum before it (passed: there was one)
            auto find = [&](double w) {
                double s = w;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, s, off);
                    if (lane >= off) s += y;
                }
                const unsigned some = __ballot_sync(0xffffffffu, w > 0.);
                const unsigned hit = __ballot_sync(0xffffffffu, w > 0. && start + s > want);
                const int k = hit ? __ffs(hit) - 1 : 31 - __clz(some);
                start += __shfl_sync(0xffffffffu, s - w, k);
                passed = hit != 0u;
                return k;
            };
            const Two t = cluster.map_shared_rank(&S, lane & (kCluster - 1))->total[(pass - 1) & 1];
            if (find(lane < kCluster ? value(t) : 0.) == rank) {
                const int w = find(lane < kWarps ? value(S.part[lane]) : 0.);
                const int i0 = piece(w), i1 = piece(w + 1), stretch = (i1 - i0 + 31) / 32;
                Two s{0.f, 0.f};
                for (int i = i0 + lane * stretch; i < min(i0 + (lane + 1) * stretch, i1); ++i) s = add(s, weight(cmd, i));
                const int j0 = i0 + find(value(s)) * stretch, j1 = min(j0 + stretch, i1);
                int x = -1;
                for (int j = j0; j < j1; j += 32) {
                    const double v = j + lane < j1 ? value(weight(cmd, j + lane)) : 0.;
                    if (!__any_sync(0xffffffffu, v > 0.)) continue;
                    const double from = start;
                    const int k = find(v);
                    x = j + k;
                    if (passed) break;
                    start = from + warp_sum(v);
                }
                if (lane == 0) A.next[b] = x;
            }
        }
    }
    // behind the path: -1
    if (tid == 0) S.n_path = n_path;
    __syncthreads();
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
    cluster.sync();  // the others may still read this CTA's sums
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
