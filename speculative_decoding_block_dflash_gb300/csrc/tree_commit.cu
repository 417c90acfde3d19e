// Moves of a drafted tree's accepted keys and values to consecutive cache positions.
//
// For s = 1 .. a the position ctx + s takes what ctx + path[s] held. The path increases strictly, so
// path[s] >= s and a position is written only after every move that reads it has been read: moves taken in
// order never read what they wrote, as position s is the source of an earlier move only. A thread owns 16
// bytes of one (layer, cache, head) column and takes that column's moves in order, eight loads in flight, then
// their stores: no move of another thread touches its column, so nothing is synchronised.
//
// The request's positions and page offsets are worked out once per CTA into shared memory. Bound: latency
// (few bytes; the load and the store are two trips to memory, after two for the path and the pages).
// Measured in replayed graphs: 4 moves in one layer (4 heads of 512) 2.9 us; 32 requests' 6 moves in 32 layers (8 heads
// of 128, 27 MB) 6.3 us where L2 holds the slots, 9.5 where it does not.
#include <algorithm>

#include "dflash_device.cuh"
#include "tree.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;

struct CommitReq {
    int32_t ctx, accepted, n, L;
    uint32_t error;  // 0, or the bit that says why the request is left as it is
};

__device__ __forceinline__ CommitReq commit_request(const TreeCommitParams& p, int32_t b)
{
    CommitReq r;
    r.L = __ldg(p.seq_lens + b);
    r.n = p.num_nodes ? __ldg(p.num_nodes + b) : p.T;
    r.accepted = __ldg(p.accepted + b);
    r.ctx = r.L - r.n;
    r.error = 0u;
    if (r.n < 0 || r.n > p.T)
        r.error = DFLASH_DEVERR_TREE;
    else if (r.n > 0 && (r.L < r.n || r.L > p.max_seq_len))
        r.error = DFLASH_DEVERR_SEQ_LEN;
    else if (r.n > 0 && (r.accepted < 0 || r.accepted >= r.n))
        r.error = DFLASH_DEVERR_TREE;
    return r;
}

// Step s of the path is sound: from 0, strictly increasing, below n.
__device__ __forceinline__ bool step_ok(const int32_t* path, int32_t s, int32_t n)
{
    const int32_t at = __ldg(path + s);
    return s == 0 ? at == 0 : at < n && at > __ldg(path + s - 1);
}

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const TreeCommitParams p, bool write_lens)
{
    __shared__ int64_t src_s[DFLASH_MAX_TREE_NODES], dst_s[DFLASH_MAX_TREE_NODES];
    const int32_t b = blockIdx.y;
    const int tid = threadIdx.x;
    const CommitReq r = commit_request(p, b);
    const int32_t* path = p.path + (int64_t)b * p.T;
    uint32_t error = r.error;
    if (!error && r.n > 0) {
        const bool ok = tid > r.accepted || step_ok(path, tid, r.n);  // accepted < n <= kThreads
        if (__syncthreads_and(ok) == 0) error = DFLASH_DEVERR_TREE;
    }
    const bool skip = error != 0u || r.n == 0;
    if (blockIdx.x == 0 && tid == 0) {
        if (error) raise_error(p.err, error);
        if (write_lens) p.new_lens[b] = skip ? r.L : r.ctx + r.accepted + 1;
    }
    if (skip || r.accepted == 0) return;
    if (tid >= 1 && tid <= r.accepted) {
        const int32_t from = r.ctx + __ldg(path + tid), to = r.ctx + tid;
        const int32_t* pages = p.page_table + (int64_t)b * p.max_pages;
        const int32_t fp = __ldg(pages + from / p.page_size), tp = __ldg(pages + to / p.page_size);
        const bool ok = fp >= 0 && fp < p.num_pages && tp >= 0 && tp < p.num_pages;
        if (!ok) raise_error(p.err, DFLASH_DEVERR_PAGE_ID);
        src_s[tid] = fp * p.sp + (int64_t)(from % p.page_size) * p.ss;
        // a node already in place, or whose page is unknown, does not move
        dst_s[tid] = ok && from != to ? tp * p.sp + (int64_t)(to % p.page_size) * p.ss : -1;
    }
    __syncthreads();
    const int32_t vecs = p.row_bytes / 16;
    const int64_t columns = (int64_t)p.layers * 2 * p.Hkv * vecs;
    for (int64_t c = (int64_t)blockIdx.x * kThreads + tid; c < columns; c += (int64_t)gridDim.x * kThreads) {
        const int32_t vec = (int32_t)(c % vecs);
        int64_t rest = c / vecs;
        const int32_t head = (int32_t)(rest % p.Hkv);
        rest /= p.Hkv;
        const int32_t layer = (int32_t)(rest >> 1);
        char* base = static_cast<char*>(rest & 1 ? p.v : p.k) + layer * p.sl + head * p.sh + vec * 16;
        for (int32_t s0 = 1; s0 <= r.accepted; s0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (s0 + u <= r.accepted && dst_s[s0 + u] >= 0)
                    x[u] = *reinterpret_cast<const uint4*>(base + src_s[s0 + u]);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (s0 + u <= r.accepted && dst_s[s0 + u] >= 0) *reinterpret_cast<uint4*>(base + dst_s[s0 + u]) = x[u];
        }
    }
}

// new_lens written over seq_lens: after the moves, which every CTA of a request derives from the old lengths.
__global__ void __launch_bounds__(kThreads) tree_commit_lens_kernel(const TreeCommitParams p)
{
    const int32_t b = blockIdx.x * kThreads + threadIdx.x;
    if (b >= p.B) return;
    const CommitReq r = commit_request(p, b);
    bool ok = r.error == 0u && r.n > 0;
    if (ok)
        for (int32_t s = 0; s <= r.accepted; ++s) ok = ok && step_ok(p.path + (int64_t)b * p.T, s, r.n);
    if (ok) p.new_lens[b] = r.ctx + r.accepted + 1;
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitParams& p, cudaStream_t stream)
{
    const bool in_place = p.new_lens == p.seq_lens;
    const int64_t columns = (int64_t)p.layers * 2 * p.Hkv * (p.row_bytes / 16);
    // a thread per column; a large batch of many layers loops, eight waves of CTAs at most
    const int64_t most = std::max<int64_t>(1, (int64_t)device_sm_count() * 8 * 8 / p.B);
    const int64_t want = (columns + kThreads - 1) / kThreads;
    tree_commit_kernel<<<dim3((unsigned)std::min(want, most), (unsigned)p.B), kThreads, 0, stream>>>(
        p, p.new_lens != nullptr && !in_place);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !in_place || !p.new_lens) return e;
    tree_commit_lens_kernel<<<(p.B + kThreads - 1) / kThreads, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dflash
