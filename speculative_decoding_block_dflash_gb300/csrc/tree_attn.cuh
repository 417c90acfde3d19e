// Device helpers of the tree attention kernels: a request's geometry, the deal of key tiles to
// ranges, and the ancestors of a tree's nodes.
#pragma once

#include <cmath>

#include "dflash_device.cuh"
#include "tree.h"

namespace dflash {

// A request as the kernels see it. nt = 0 when there is nothing to attend to (no nodes, or a bad length or
// tree size, which sets `bad`).
struct TreeReq {
    int32_t n, ctx, L, lo;  // nodes, context keys, keys, first key that any node sees
    int32_t tile0, nt;      // first key tile and number of them
    bool bad;
};

__device__ __forceinline__ TreeReq tree_request(const TreeAttnParams& p, int32_t b)
{
    TreeReq r;
    r.n = p.num_nodes ? __ldg(p.num_nodes + b) : p.T;
    r.L = __ldg(p.seq_lens + b);
    const bool bad_n = r.n < 0 || r.n > p.T;
    const bool bad_l = !bad_n && r.n > 0 && (r.L < r.n || r.L > p.max_seq_len);
    r.bad = bad_n || bad_l;
    r.ctx = r.L - r.n;
    r.lo = p.window > 0 ? max(0, r.ctx - p.window + 1) : 0;
    if (r.bad || r.n == 0) {
        r.tile0 = r.nt = 0;
        return r;
    }
    r.tile0 = r.lo / p.tile;
    r.nt = (r.L + p.tile - 1) / p.tile - r.tile0;
    return r;
}

__device__ __forceinline__ uint32_t tree_request_error(const TreeAttnParams& p, const TreeReq& r)
{
    if (!r.bad) return 0u;
    return (r.n < 0 || r.n > p.T) ? DFLASH_DEVERR_TREE : DFLASH_DEVERR_SEQ_LEN;
}

// The deal counts in units of a key tile's time. A pair of nt tiles weighs pair_cost + nt: its first units stand for
// loading its queries, filling the pipeline and writing its result, so that ranges of many short pairs get fewer
// tiles.
__device__ __forceinline__ int64_t tree_weight(const TreeAttnParams& p, const TreeReq& r)
{
    return r.nt > 0 ? r.nt + p.pair_cost : 0;
}

// Weight of all (request, KV head) pairs before request b (b = B: of all). Called by a whole warp.
__device__ __forceinline__ int64_t tree_weight_before(const TreeAttnParams& p, int32_t b_end)
{
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
#pragma unroll 1
    for (int32_t b = lane; b < b_end; b += 32) sum += tree_weight(p, tree_request(p, b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    return sum * p.Hkv;
}

// Ranges in use: none has weight 0, so that a pair's partials lie in consecutive ranges.
__device__ __forceinline__ int32_t ranges_used(const TreeAttnParams& p, int64_t total)
{
    return (int32_t)(total < p.ranges ? total : p.ranges);
}

// a / b for a >= 0, b > 0; the 64-bit division is a long routine, and the numbers are mostly small.
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b)
{
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Where range r begins when a weight of `total` is dealt to `ranges` ranges.
__device__ __forceinline__ int64_t range_begin(int64_t total, int32_t ranges, int32_t r)
{
    return div_small(total * r, ranges);
}

// The range that holds unit x of the weight.
__device__ __forceinline__ int32_t range_of(int64_t total, int32_t ranges, int64_t x)
{
    int32_t r = (int32_t)div_small(x * ranges, total);
    while (r + 1 < ranges && range_begin(total, ranges, r + 1) <= x) ++r;
    while (r > 0 && range_begin(total, ranges, r) > x) --r;
    return r;
}

// A walk over the pieces of one range: a piece is the part of one (request, KV head) pair's tiles that lies in it.
struct PieceWalk {
    int64_t left;      // weight of the range still to come, this piece's part included
    int32_t b, g, at;  // the pair (b, g), and where in its weight the piece begins
    int32_t t0, t1;    // the piece: tiles [t0, t1) of the pair's
    TreeReq req;

    __device__ __forceinline__ void cut(const TreeAttnParams& p)
    {
        const int64_t weight = tree_weight(p, req);
        const int64_t end = left < weight - at ? at + left : weight;
        t0 = max(0, at - p.pair_cost);
        t1 = max(0, (int32_t)end - p.pair_cost);
        left -= end - at;
    }
    __device__ __forceinline__ bool done() const { return t1 <= t0; }
    // Start of range r (a whole warp calls it).
    __device__ __forceinline__ void start(const TreeAttnParams& p, int32_t r)
    {
        const int lane = threadIdx.x & 31;
        b = g = at = t0 = t1 = 0;
        left = 0;
        req.n = req.ctx = req.L = req.lo = req.tile0 = req.nt = 0;
        req.bad = false;
        // the first 32 requests, a lane each: all there are, mostly
        const TreeReq own = lane < p.B ? tree_request(p, lane) : req;
        int64_t mine = tree_weight(p, own) * p.Hkv;
        int64_t total = mine;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
        if (p.B > 32) total = tree_weight_before(p, p.B);
        const int32_t used = ranges_used(p, total);
        int64_t x = 0;
        if (r < used) {
            x = range_begin(total, used, r);
            left = range_begin(total, used, r + 1) - x;
        }
        if (left <= 0) return;
#pragma unroll 1
        for (int32_t b0 = 0;; b0 += 32) {
            if (b0 > 0) mine = b0 + lane < p.B ? tree_weight(p, tree_request(p, b0 + lane)) * p.Hkv : 0;
            int64_t incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, x < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b = b0 + src;
                x -= __shfl_sync(0xffffffffu, incl - mine, src);
                break;
            }
            x -= __shfl_sync(0xffffffffu, incl, 31);
            if (b0 + 32 >= p.B) {  // not reached: x lies below the total
                left = 0;
                return;
            }
        }
        if (b < 32) {
            req.n = __shfl_sync(0xffffffffu, own.n, b);
            req.L = __shfl_sync(0xffffffffu, own.L, b);
            req.ctx = __shfl_sync(0xffffffffu, own.ctx, b);
            req.lo = __shfl_sync(0xffffffffu, own.lo, b);
            req.tile0 = __shfl_sync(0xffffffffu, own.tile0, b);
            req.nt = __shfl_sync(0xffffffffu, own.nt, b);
        } else {
            req = tree_request(p, b);
        }
        g = (int32_t)div_small(x, tree_weight(p, req));
        at = (int32_t)(x - g * tree_weight(p, req));
        cut(p);
        if (done()) next(p);  // the range begins in a pair's first units and ends there, or it does not reach a tile
    }
    // The next piece that holds a tile, if any (done() otherwise).
    __device__ __forceinline__ void next(const TreeAttnParams& p)
    {
        t0 = t1 = 0;
        while (left > 0 && t1 <= t0) {
            at = 0;
            if (++g == p.Hkv) {
                g = 0;
                do {
                    if (++b >= p.B) {  // not reached: the range lies below the total
                        left = 0;
                        return;
                    }
                    req = tree_request(p, b);
                } while (req.nt == 0);
            }
            cut(p);
        }
    }
    // Whether the piece is a whole pair (its result is final), and its partial's slot otherwise: the pair's
    // first piece takes slot 1, a later one slot 0 (a range holds at most one of each that is not whole).
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == req.nt; }
    __device__ __forceinline__ int slot() const { return t0 == 0 ? 1 : 0; }
};

// Query tile `sub` of a pair: heads gc, node tile rt and slice dv of the value's dims.
struct SubTile {
    int32_t gc, rt, dv;
};

__device__ __forceinline__ SubTile sub_tile(const TreeAttnParams& p, int32_t sub)
{
    SubTile s;
    const int32_t odd = p.pair ? sub & 1 : 0;
    if (p.pair) sub >>= 1;
    const int32_t tiles = p.pair ? p.nrt / 2 : p.nrt;
    s.dv = sub % p.ndv;
    const int32_t rest = sub / p.ndv;
    s.rt = rest % tiles;
    if (p.pair) s.rt = 2 * s.rt + odd;
    s.gc = rest / tiles;
    return s;
}

__device__ __forceinline__ int64_t tree_part_row(const TreeAttnParams& p, int32_t range, int32_t sub, int slot)
{
    return (((int64_t)range * p.n_sub + sub) * 2 + slot) * p.rows;
}

// What a row is scaled by, and its lse. A partial without a visible key has a sum of 0 and is all zeros, with lse -inf. A
// row that has seen all of its keys, its own among them, has a sum of 0 only if every score was -inf: it is NaN, as one
// with a score of NaN or +inf is, whose sum is NaN.
__device__ __forceinline__ float tree_inv_sum(float sum, bool all_keys)
{
    if (sum != 0.f) return 1.f / sum;
    return all_keys ? NAN : 0.f;
}

__device__ __forceinline__ float tree_row_lse(float lse, float sum, bool all_keys)
{
    if (sum != 0.f) return lse;
    return all_keys ? NAN : -INFINITY;
}

// The larger value; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Parent of node i as the kernels use it: -1 where the table holds none or something out of range.
__device__ __forceinline__ int32_t tree_parent(const int32_t* parents, int32_t i, uint32_t* err)
{
    const int32_t a = __ldg(parents + i);
    if (a >= -1 && a < i) return a;
    raise_error(err, DFLASH_DEVERR_TREE);
    return -1;
}

// What the nodes [node0, node0 + count) of a tree see, in two steps with a barrier of the calling threads
// between them. par_s[T] takes the parents; then anc_s[i * words + w] takes the nodes that node0 + i sees
// (bit j of word w is node 32 w + j) and lo_s[i] the first context key that it sees. A node walks
// up to the root: as a parent comes before its children the walk ends, whatever the table holds.
__device__ __forceinline__ void tree_load_parents(const TreeAttnParams& p, int32_t b, int32_t n, int32_t* par_s,
                                                  int tid, int nthreads)
{
    for (int32_t i = tid; i < n; i += nthreads) par_s[i] = tree_parent(p.parents + (int64_t)b * p.T, i, p.err);
}

__device__ __forceinline__ void tree_walk_nodes(const TreeAttnParams& p, const TreeReq& r, int32_t node0, int32_t count,
                                                const int32_t* par_s, uint32_t* anc_s, int32_t* lo_s, int tid,
                                                int nthreads)
{
    const int words = (p.T + 31) / 32;
    for (int32_t i = tid; i < count; i += nthreads) {
        for (int w = 0; w < words; ++w) anc_s[i * words + w] = 0u;
        int32_t depth = -1;
        if (node0 + i < r.n) {
            for (int32_t j = node0 + i; j >= 0; j = par_s[j]) {
                ++depth;
                // an ancestor `depth` levels up stands `depth` positions back
                if (p.window == 0 || depth < p.window) anc_s[i * words + (j >> 5)] |= 1u << (j & 31);
            }
        }
        lo_s[i] = p.window > 0 ? max(0, r.ctx + depth - p.window + 1) : 0;
    }
}

}  // namespace dflash
