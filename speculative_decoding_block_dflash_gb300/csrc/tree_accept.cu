// Longest accepted path of drafted trees: the target's token at every node (argmax of its row of logits, the
// smallest id among equal maxima) and the walk from the root along the drafted tokens that agree.
//
// The argmax is one stream over the real nodes' rows; padding rows are not read. The rows of all requests, laid
// end to end, are cut into equal parts, one CTA each, four CTAs an SM (one wave): a CTA streams its part, four
// to eight 16-byte loads in flight per thread, and settles a row where it ends. (A CTA per 64 KB of a row spent
// a third of its life in its first load's latency and in the arrival at its end: 53 us for 452 rows of 262144
// bf16 logits, which take 45 now, 5.3 TB/s.) A thread keeps (maximum, first id) in increasing id order, then forms a 64-bit key, the
// order-preserving image of the value above the complement of the id, so that the largest key is the largest
// logit of smallest id; -0 is taken as +0 first, so equal values have equal images. CTAs merge a row's keys
// with a 64-bit atomicMax, whose result does not depend on the order.
//
// Each CTA adds what it has read of a request's logits to the request's counter; the one that completes it (no
// waiting) reads its rows' keys. Every node whose token is its parent's target token offers itself to the
// parent with an atomicMin in shared memory, so each node knows its first agreeing child, and one thread
// follows those links. The keys and the counters are left at zero.
#include <algorithm>

#include "tree_attn.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;
constexpr int kCtasPerSm = 4;
constexpr int kPartBytes = 8192;  // a CTA's part is this long at least

__device__ __forceinline__ unsigned long long make_key(float x, uint32_t id)
{
    uint32_t u = __float_as_uint(x + 0.f);  // -0 -> +0
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((unsigned long long)u << 32) | (0xFFFFFFFFu - id);
}

template <typename E>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void widen(const uint4& w, float (&x)[8])
    {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float largest(const uint4& w)
    {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16* r, int64_t i) { return __bfloat162float(r[i]); }
};
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void widen(const uint4& w, float (&x)[4])
    {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float largest(const uint4& w)
    {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                     fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    static __device__ __forceinline__ float one(const float* r, int64_t i) { return r[i]; }
};

__device__ __forceinline__ int32_t nodes_of(const TreeAcceptParams& p, int32_t b, bool& bad)
{
    const int32_t n = p.num_nodes ? __ldg(p.num_nodes + b) : p.T;
    bad = n < 0 || n > p.T;
    return bad ? 0 : n;
}

template <typename E>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) tree_accept_kernel(const TreeAcceptParams p)
{
    using V = Vec<E>;
    __shared__ unsigned long long warp_best[kThreads / 32];
    __shared__ int64_t sh_rows, sh_first;
    __shared__ int32_t sh_b, last;
    __shared__ int32_t tok_s[DFLASH_MAX_TREE_NODES], next_s[DFLASH_MAX_TREE_NODES];
    const int tid = threadIdx.x, lane = tid & 31;
    bool bad;

    // requests of no nodes have their answer at once
    for (int32_t b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (nodes_of(p, b, bad) != 0) continue;
        if (tid == 0) {
            if (bad) raise_error(p.err, DFLASH_DEVERR_TREE);
            p.accepted[b] = 0;
            p.next_token[b] = -1;
        }
        for (int32_t i = tid; i < p.T; i += kThreads) {
            p.path[(int64_t)b * p.T + i] = -1;
            if (p.target_argmax) p.target_argmax[(int64_t)b * p.T + i] = -1;
        }
    }
    // This CTA's part of the logits: [at, end) of the real rows laid end to end; where it begins.
    if (tid < 32) {
        int64_t rows = 0;
        for (int32_t b = lane; b < p.B; b += 32) rows += nodes_of(p, b, bad);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, off);
        // rows * V <= 2^47 and gridDim.x < 2^12
        const int64_t first = rows * p.V * blockIdx.x / gridDim.x;
        int64_t row = first / p.V;
        for (int32_t b0 = 0; b0 < p.B; b0 += 32) {
            const int32_t n = b0 + lane < p.B ? nodes_of(p, b0 + lane, bad) : 0;
            int32_t incl = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, row < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const int32_t before = __shfl_sync(0xffffffffu, incl - n, src);
                if (lane == 0) {
                    sh_b = b0 + src;
                    sh_first = first - (first / p.V - (row - before)) * p.V;  // from the request's own first logit
                    sh_rows = rows;
                }
                break;
            }
            row -= __shfl_sync(0xffffffffu, incl, 31);
            if (b0 + 32 >= p.B && lane == 0) sh_rows = 0;  // no rows at all
        }
    }
    __syncthreads();
    if (sh_rows == 0) return;
    int64_t left = sh_rows * p.V * (blockIdx.x + 1) / gridDim.x - sh_rows * p.V * blockIdx.x / gridDim.x;
    int32_t b = sh_b;
    int64_t at = sh_first;  // in request b's logits
    while (left > 0) {
        const int32_t n = nodes_of(p, b, bad);
        if (n == 0) {
            ++b;
            continue;
        }
        int64_t taken = 0;  // of request b's logits by this CTA
        while (left > 0 && at < (int64_t)n * p.V) {
            // a row, or the part of it that is this CTA's: ids [e0, e1), in vectors from a 16-byte boundary on. A cut
            // inside a row is moved up to the next boundary, by both its sides alike.
            const int32_t node = (int32_t)(at / p.V);
            const int32_t e0 = (int32_t)(at - (int64_t)node * p.V);
            const int32_t e1 = (int32_t)min((int64_t)p.V, e0 + left);
            const E* r = static_cast<const E*>(p.logits) + ((int64_t)b * p.T + node) * p.row_stride;
            const int32_t mis = (int32_t)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(E));
            const int32_t vecs = (int32_t)(((int64_t)p.V + mis + V::kN - 1) / V::kN);
            const int32_t q0 = e0 == 0 ? 0 : (int32_t)(((int64_t)e0 + mis + V::kN - 1) / V::kN);
            const int32_t q1 = e1 == p.V ? vecs : (int32_t)(((int64_t)e1 + mis + V::kN - 1) / V::kN);
            const E* base = r - mis;
            float bv = -INFINITY;
            int32_t bi = -1;
            auto take = [&](float x, int32_t id) {
                const bool more = x > bv || bi < 0;
                bv = more ? x : bv;
                bi = more ? id : bi;
            };
            auto take_vec = [&](const uint4& w, int32_t id) {
                // a vector whose largest value does not exceed the running one (nearly all) costs four maxima
                const float most = V::largest(w);
                if (!(most > bv || bi < 0)) return;
                float x[V::kN];
                V::widen(w, x);
                int first = 0;
#pragma unroll
                for (int e = V::kN - 1; e >= 0; --e)
                    if (x[e] == most) first = e;
                bv = most;
                bi = id + first;
            };
            auto id_of = [&](int32_t q) { return (int32_t)((uint32_t)q * V::kN - mis); };
            // vectors at the row's ends that hold other elements too are read element by element
            const int32_t whole0 = mis ? 1 : 0, whole1 = (int32_t)(((int64_t)p.V + mis) / V::kN);
            auto take_part = [&](int32_t q) {
                for (int e = 0; e < V::kN; ++e) {
                    const int64_t id = (int64_t)q * V::kN - mis + e;
                    if (id >= 0 && id < p.V) take(V::one(r, id), (int32_t)id);
                }
            };
            auto load = [&](int32_t q) { return __ldcs(reinterpret_cast<const uint4*>(base) + q); };
            int32_t q = q0 + tid;
            if (q < q1 && q < whole0) {
                take_part(q);
                q += kThreads;
            }
            const int32_t qw = min(q1, whole1);
            uint4 cur[kBatch], nxt[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (q + u * kThreads < qw) cur[u] = load(q + u * kThreads);
#pragma unroll 1
            while (q + (2 * kBatch - 1) * kThreads < qw) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) nxt[u] = load(q + (kBatch + u) * kThreads);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) take_vec(cur[u], id_of(q + u * kThreads));
#pragma unroll
                for (int u = 0; u < kBatch; ++u) cur[u] = nxt[u];
                q += kBatch * kThreads;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (q + (kBatch + u) * kThreads < qw) nxt[u] = load(q + (kBatch + u) * kThreads);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (q + u * kThreads < qw) take_vec(cur[u], id_of(q + u * kThreads));
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (q + (kBatch + u) * kThreads < qw) take_vec(nxt[u], id_of(q + (kBatch + u) * kThreads));
            while (q < qw) q += kThreads;
            if (q < q1) take_part(q);  // the last vector, if it is not whole
            unsigned long long best = bi >= 0 ? make_key(bv, (uint32_t)bi) : 0ull;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
            if (lane == 0) warp_best[tid >> 5] = best;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kThreads / 32; ++w) best = max(best, warp_best[w]);
                if (best) atomicMax(p.keys + (int64_t)b * p.T + node, best);
            }
            __syncthreads();
            taken += e1 - e0;
            left -= e1 - e0;
            at += e1 - e0;
        }
        if (tid == 0) {
            __threadfence();
            const unsigned long long all = (unsigned long long)n * p.V;
            last = atomicAdd(p.counters + b, (unsigned long long)taken) + taken == all;
        }
        __syncthreads();
        if (last) {
            __threadfence();
            const int64_t row0 = (int64_t)b * p.T;
            for (int32_t i = tid; i < p.T; i += kThreads) {
                int32_t tok = -1;
                if (i < n) {
                    const unsigned long long key = atomicExch(p.keys + row0 + i, 0ull);
                    tok = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
                    tok_s[i] = tok;
                    next_s[i] = n;
                }
                if (p.target_argmax) p.target_argmax[row0 + i] = tok;
            }
            __syncthreads();
            for (int32_t i = tid; i < n; i += kThreads) {
                const int32_t a = tree_parent(p.parents + row0, i, p.err);
                if (a >= 0 && __ldg(p.tokens + row0 + i) == tok_s[a]) atomicMin(next_s + a, i);
            }
            __syncthreads();
            if (tid == 0) {
                int32_t len = 0, node = 0;
                p.path[row0] = 0;
                while (next_s[node] < n) {
                    node = next_s[node];
                    p.path[row0 + ++len] = node;
                }
                p.accepted[b] = len;
                p.next_token[b] = tok_s[node];
                p.counters[b] = 0ull;
                last = len;
            }
            __syncthreads();
            for (int32_t i = last + 1 + tid; i < p.T; i += kThreads) p.path[row0 + i] = -1;
        }
        __syncthreads();
        ++b;
        at = 0;
    }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptParams& p, cudaStream_t stream)
{
    // one wave of equal parts, or fewer of 8 KB
    const int64_t bytes = (int64_t)p.B * p.T * p.V * (p.dtype == DFLASH_BF16 ? 2 : 4);
    const int64_t wave = (int64_t)kCtasPerSm * device_sm_count();
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min(wave, bytes / kPartBytes));
    if (p.dtype == DFLASH_BF16)
        tree_accept_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
    else
        tree_accept_kernel<float><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dflash
