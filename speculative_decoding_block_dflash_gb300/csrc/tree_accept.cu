// Longest accepted path of drafted trees: the target's token at every node (argmax of its row of logits, the
// smallest id among equal maxima) and the walk from the root along the drafted tokens that agree.
//
// The argmax is one stream over the real nodes' rows; padding rows are not read. A row is cut into slices of
// about 64 KB, one CTA each, eight 16-byte loads in flight per thread. A thread keeps (maximum, first id) in
// increasing id order, then forms a 64-bit key, the order-preserving image of the value above
// the complement of the id, so that the largest key is the largest logit of smallest id; -0 is taken as +0 first,
// so equal values have equal images. CTAs merge a row's keys with a 64-bit atomicMax, whose result does
// not depend on the order.
//
// The last CTA of a request to arrive (a counter, no waiting) reads its rows' keys. Every node whose token is its parent's
// target token offers itself to the parent with an atomicMin in shared memory, so each node knows
// its first agreeing child, and one thread follows those links. The keys and the counter are left at zero.
#include <algorithm>

#include "tree_attn.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;
constexpr int kCtasPerSm = 4;
constexpr int kSliceBytes = 65536;

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
    static __device__ __forceinline__ float one(const float* r, int64_t i) { return r[i]; }
};

template <typename E>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) tree_accept_kernel(const TreeAcceptParams p, int32_t slices)
{
    using V = Vec<E>;
    __shared__ unsigned long long warp_best[kThreads / 32];
    __shared__ int32_t last;
    __shared__ int32_t tok_s[DFLASH_MAX_TREE_NODES], next_s[DFLASH_MAX_TREE_NODES];
    const int tid = threadIdx.x;
    const int32_t b = blockIdx.y / p.T, node = blockIdx.y % p.T;
    int32_t n = p.num_nodes ? __ldg(p.num_nodes + b) : p.T;
    const bool bad = n < 0 || n > p.T;
    if (bad) n = 0;
    if (n == 0) {
        if (node == 0 && blockIdx.x == 0) {
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
        return;
    }
    if (node >= n) return;

    // Slices are cut at the row's 16-byte boundaries, counted from the one at or before its first element;
    // the vectors at the row's two ends that hold other elements too are read element by element.
    const E* r = static_cast<const E*>(p.logits) + (int64_t)blockIdx.y * p.row_stride;
    const int32_t mis = (int32_t)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(E));
    const int64_t vecs = ((int64_t)p.V + mis + V::kN - 1) / V::kN;
    const int64_t per = (vecs + slices - 1) / slices;
    const int64_t q0 = blockIdx.x * per, q1 = min(vecs, q0 + per);
    float bv = -INFINITY;
    int64_t bi = -1;
    auto take = [&](float x, int64_t id) {
        const bool more = x > bv || bi < 0;
        bv = more ? x : bv;
        bi = more ? id : bi;
    };
    auto take_vec = [&](const uint4& w, int64_t q) {
        float x[V::kN];
        V::widen(w, x);
#pragma unroll
        for (int e = 0; e < V::kN; ++e) take(x[e], q * V::kN - mis + e);
    };
    auto whole = [&](int64_t q) { return q * V::kN >= mis && (q + 1) * V::kN - mis <= p.V; };
    auto load = [&](int64_t q) { return __ldcs(reinterpret_cast<const uint4*>(r + (q * V::kN - mis))); };
    int64_t q = q0 + tid;
    if (q < q1 && !whole(q)) {  // the row's first vector (or its only one)
        for (int e = 0; e < V::kN; ++e) {
            const int64_t id = q * V::kN - mis + e;
            if (id >= 0 && id < p.V) take(V::one(r, id), id);
        }
        q += kThreads;
    }
    for (; q + (int64_t)(kBatch - 1) * kThreads < q1 && whole(q + (int64_t)(kBatch - 1) * kThreads);
         q += (int64_t)kBatch * kThreads) {
        uint4 w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) w[u] = load(q + u * kThreads);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) take_vec(w[u], q + u * kThreads);
    }
    for (; q < q1; q += kThreads) {
        if (whole(q)) {
            take_vec(load(q), q);
        } else {
            for (int e = 0; e < V::kN; ++e) {
                const int64_t id = q * V::kN - mis + e;
                if (id >= 0 && id < p.V) take(V::one(r, id), id);
            }
        }
    }
    unsigned long long best = bi >= 0 ? make_key(bv, (uint32_t)bi) : 0ull;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
    if ((tid & 31) == 0) warp_best[tid >> 5] = best;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kThreads / 32; ++w) best = max(best, warp_best[w]);
        if (best) atomicMax(p.keys + blockIdx.y, best);
        __threadfence();
        last = atomicAdd(p.counters + b, 1) == n * slices - 1;
    }
    __syncthreads();
    if (!last) return;

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
        int32_t len = 0, at = 0;
        p.path[row0] = 0;
        while (next_s[at] < n) {
            at = next_s[at];
            p.path[row0 + ++len] = at;
        }
        p.accepted[b] = len;
        p.next_token[b] = tok_s[at];
        p.counters[b] = 0;
        last = len;
    }
    __syncthreads();
    for (int32_t i = last + 1 + tid; i < p.T; i += kThreads) p.path[row0 + i] = -1;
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptParams& p, cudaStream_t stream)
{
    const int64_t row_bytes = (int64_t)p.V * (p.dtype == DFLASH_BF16 ? 2 : 4);
    const int64_t rows = (int64_t)p.B * p.T;
    // slices of 64 KB, shorter ones (8 KB at least) while they leave the GPU's first wave part empty
    int64_t slices = std::max<int64_t>(1, (row_bytes + kSliceBytes - 1) / kSliceBytes);
    const int64_t wave = (int64_t)kCtasPerSm * device_sm_count();
    if (rows * slices < wave) slices = std::max(slices, std::min(wave / rows, (row_bytes + 8191) / 8192));
    // the arrival counter holds T * slices
    slices = std::min<int64_t>(slices, 65535);
    const dim3 grid((unsigned)slices, (unsigned)rows);
    if (p.dtype == DFLASH_BF16)
        tree_accept_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p, (int32_t)slices);
    else
        tree_accept_kernel<float><<<grid, kThreads, 0, stream>>>(p, (int32_t)slices);
    return cudaGetLastError();
}

}  // namespace dflash
