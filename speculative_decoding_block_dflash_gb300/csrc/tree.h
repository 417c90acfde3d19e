// Internal interface of the tree operators: the C-ABI front end (tree_api.cpp) and the kernels.
// Not installed; not part of the ABI.
#pragma once

#include "dflash_internal.h"

namespace dflash {

// One dflash_tree_attn call, validated on the host.
//
// Work. A query tile is the rows of npt nodes x Gc heads of one KV head (row = node * Gc + head, `rows` of
// them); a request has n_sub = (G / Gc) * nrt * ndv of them, nrt being the node tiles, per KV head, ndv being
// the slices of the value's dims that one CTA's accumulators hold. Every one of them reads the same K/V, so the
// key tiles of all (request, KV head) pairs, laid end to end, are cut into `ranges` equal ranges and a CTA
// takes (range, query tile): each range is streamed by the n_sub CTAs of consecutive block numbers at about the
// same time, out of L2 but for the first. A range may hold the end of one pair's keys, whole pairs, and the
// start of another's: whatever the lengths, every CTA streams the same number of key tiles to within one. A
// pair that lies in several ranges leaves one normalised partial per range, and the join kernel merges them by
// their log-sum-exp.
struct TreeAttnParams {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* parents;    // [B, T]
    const int32_t* num_nodes;  // [B] or nullptr
    void* out;
    float* lse;
    uint32_t* err;
    float* part_out;  // [ranges][n_sub][2 slots][rows][DV]
    float* part_lse;  // [ranges][n_sub][2 slots][rows]
    int32_t B, T, Hq, Hkv, G, D;
    int32_t page_size, num_pages, max_pages, max_seq_len;
    int64_t sp, ss, sh;
    int32_t window;
    float scale;
    int32_t dtype;
    int32_t Gc, npt, nrt, ndv, rows, DV, n_sub, ranges;
    int32_t pair;  // 1: tensor-core CTA pairs; neighbouring node tiles are neighbouring query tiles
    int32_t tile;  // keys per tile
    int32_t pair_cost;  // of a pair beside its tiles, in tiles
    unsigned long long wait_ns;
};

// The CUDA-core kernel's 64-dim chunks for head_dim D (1, 2, 4 or 8), and the CTAs of it that an SM holds with query
// tiles of `rows`: its registers are bounded to that.
constexpr int simt_chunks(int D) { return D <= 64 ? 1 : D <= 128 ? 2 : D <= 256 ? 4 : 8; }
constexpr int simt_ctas_per_sm(int D, int rows)
{
    return rows <= 16 ? (D <= 128 ? 3 : 2) : rows <= 32 ? (D <= 128 ? 2 : 1) : (D <= 64 ? 2 : 1);
}

// The query tile shape and the number of ranges of a call, for the kernel `kernel` (DFLASH_KERNEL_SIMT or _TC).
void tree_attn_plan(TreeAttnParams& p, int kernel);
bool tree_tc_supports(const dflash_dims* d);
cudaError_t launch_tree_attn_simt(const TreeAttnParams& p, cudaStream_t stream);
cudaError_t launch_tree_attn_tc(TreeAttnParams& p, cudaStream_t stream);  // may take fewer ranges than planned
cudaError_t launch_tree_join(const TreeAttnParams& p, cudaStream_t stream);
// Address of the library's own error word on the current device; dflash_read_error may clear the block behind it.
cudaError_t shared_error_word(uint32_t** word);

// Log probabilities (csrc/token_logprobs.cu).
struct LogprobsParams {
    const void* logits;
    int32_t dtype, R, V;
    int64_t row_stride;
    float temperature;
    const int32_t* tokens;
    int32_t m;  // given tokens per row
    float* token_logp;
    float* log_z;
    float* entropy;
    int32_t k;
    int32_t* top_tokens;
    float* top_logp;
    uint32_t* err;
    int32_t* counters;         // [65536]
    float* part_stat;          // [R][slices][4]
    unsigned long long* part_key;  // [R][slices][k]
    int32_t slices;
};
int32_t logprobs_slices(int32_t R, int32_t V);
cudaError_t launch_token_logprobs(const LogprobsParams& p, cudaStream_t stream);

// Longest accepted path (csrc/tree_accept.cu).
struct TreeAcceptParams {
    const void* logits;
    int32_t dtype, B, T, V;
    int64_t row_stride;
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* num_nodes;
    int32_t* accepted;
    int32_t* path;
    int32_t* next_token;
    int32_t* target_argmax;
    uint32_t* err;
    unsigned long long* keys;  // [B * T], zero between calls
    unsigned long long* counters;  // [B], zero between calls
};
cudaError_t launch_tree_accept(const TreeAcceptParams& p, cudaStream_t stream);

// Moves of accepted keys and values (csrc/tree_commit.cu).
struct TreeCommitParams {
    void* k;
    void* v;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* path;
    const int32_t* accepted;
    const int32_t* num_nodes;
    int32_t* new_lens;
    uint32_t* err;
    int32_t B, T, layers, Hkv, row_bytes;  // row_bytes: one head's dims
    int32_t page_size, num_pages, max_pages, max_seq_len;
    int64_t sp, ss, sh, sl;  // strides in bytes
};
cudaError_t launch_tree_commit(const TreeCommitParams& p, cudaStream_t stream);

}  // namespace dflash
