// C-ABI front end of the tree operators: host-side validation, plans, workspace carve-up and
// launches. See include/dflash_attn.h for the contract of each entry point.
#include <algorithm>
#include <cmath>

#include "tree.h"

namespace dflash {
namespace {

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
void clear_error() { report_error(DFLASH_OK, "%s", ""); }
dflash_status cuda_fail(cudaError_t e, const char* what)
{
    return report_error(DFLASH_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int32_t max_len_of(const dflash_dims* d)
{
    const int32_t cap = d->max_pages * d->page_size;
    return d->max_seq_len ? std::min(d->max_seq_len, cap) : cap;
}

// Fixed blocks of the workspaces: a counter per possible row or request, wherever a call's own sizes end,
// so that a workspace zeroed once serves calls of any size.
constexpr size_t kCounterBytes = 65536 * sizeof(int32_t);
constexpr size_t kKeyBytes = 65536 * sizeof(unsigned long long);

struct LogprobsLayout {
    size_t stat_off, key_off, total;
};

LogprobsLayout logprobs_layout(int32_t R, int32_t slices, int32_t k)
{
    LogprobsLayout w;
    w.stat_off = kCounterBytes;
    w.key_off = w.stat_off + round_up((size_t)R * slices * 4 * sizeof(float), 256);
    w.total = w.key_off + round_up((size_t)R * slices * k * sizeof(unsigned long long), 256);
    return w;
}

struct TreeAttnLayout {
    size_t lse_off, out_off, total;
};

TreeAttnLayout tree_attn_layout(const TreeAttnParams& p)
{
    // nothing is split when every query tile has but one range
    const size_t rows = p.ranges > 1 ? (size_t)p.ranges * p.n_sub * 2 * p.rows : 0;
    TreeAttnLayout w;
    w.lse_off = 256 + DFLASH_COUNTER_BYTES;  // (dflash_read_error clears as much after a timeout)
    w.out_off = w.lse_off + round_up(rows * sizeof(float), 256);
    w.total = w.out_off + round_up(rows * p.DV * sizeof(float), 256);
    return w;
}

void fill_sizes(TreeAttnParams& p, const dflash_dims* d, int32_t T)
{
    p.B = d->batch;
    p.T = T;
    p.Hq = d->num_q_heads;
    p.Hkv = d->num_kv_heads;
    p.G = d->num_q_heads / d->num_kv_heads;
    p.D = d->head_dim;
    p.page_size = d->page_size;
    p.num_pages = d->num_pages;
    p.max_pages = d->max_pages;
    p.max_seq_len = max_len_of(d);
    p.sp = d->kv_stride_page;
    p.ss = d->kv_stride_slot;
    p.sh = d->kv_stride_head;
    p.dtype = d->dtype;
}

}  // namespace

void tree_attn_plan(TreeAttnParams& p, int kernel)
{
    const bool tc = kernel == DFLASH_KERNEL_TC;
    const int32_t most = tc ? 128 : 64;  // rows of a query tile
    p.Gc = 1;
    for (int32_t gc = std::min(p.G, most); gc >= 1; --gc)
        if (p.G % gc == 0) {
            p.Gc = gc;
            break;
        }
    const int32_t fit = most / p.Gc;
    p.nrt = (p.T + fit - 1) / fit;
    // Several node tiles on the tensor cores: CTA pairs, an even number of tiles. Of up to 64 dims, where a pair's MMAs
    // are half empty, an odd number stays as it is (4 requests of 4k to 9k keys, 32/8 heads of 64: 90 nodes, 3 tiles,
    // 55 us against 66 in pairs; 128 nodes, 4 tiles, 72 against 68; of 128 dims and more pairs take 0.7 to 0.9 of the
    // time for 3 tiles too).
    p.pair = tc && p.nrt > 1 && (p.D > 64 || p.nrt % 2 == 0) ? 1 : 0;
    if (p.pair) p.nrt = (p.nrt + 1) / 2 * 2;
    p.npt = (p.T + p.nrt - 1) / p.nrt;  // node tiles of equal size
    p.rows = p.npt * p.Gc;
    p.tile = tc ? 128 : 64;
    // A pair's fixed cost: some 4 us, of tiles of about 1 us on the tensor cores and of rows x dims / 2500 us on the
    // CUDA cores (fp32, 8 requests of 150 keys, 26 nodes, 32/4 heads of 512: 184 us with 4 tiles, 164 with none).
    p.pair_cost = tc ? 4 : std::min(4, 10000 / (std::max(16, p.rows) * p.D));
    p.DV = !tc ? p.D : p.D <= 64 && !p.pair ? 64 : p.D <= 128 ? 128 : 256;
    p.ndv = (p.D + p.DV - 1) / p.DV;
    p.n_sub = (p.G / p.Gc) * p.nrt * p.ndv;
    // one wave: the tensor-core kernel holds one CTA per SM
    const int32_t ctas = device_sm_count() * (tc ? 1 : simt_ctas_per_sm(64 * simt_chunks(p.D), p.rows));
    p.ranges = std::max(1, ctas / p.n_sub);
}

}  // namespace dflash

using namespace dflash;

namespace {

// The kernel a call runs, or a negative status.
int tree_attn_kernel(const dflash_dims* d, int32_t requested)
{
    if (requested == DFLASH_KERNEL_SIMT) return DFLASH_KERNEL_SIMT;
    if (requested != DFLASH_KERNEL_AUTO && requested != DFLASH_KERNEL_TC) return -DFLASH_ERR_INVALID_ARG;
    if (d->dtype == DFLASH_BF16 && tree_tc_supports(d)) return DFLASH_KERNEL_TC;
    return requested == DFLASH_KERNEL_TC ? -DFLASH_ERR_UNSUPPORTED : DFLASH_KERNEL_SIMT;
}

}  // namespace

extern "C" {

size_t dflash_tree_attn_workspace_bytes(const dflash_dims* dims, int32_t max_nodes)
{
    clear_error();
    if (check_attn_dims(dims, max_nodes, DFLASH_MAX_TREE_NODES, 1) != DFLASH_OK) return 0;
    TreeAttnParams p{};
    fill_sizes(p, dims, max_nodes);
    tree_attn_plan(p, DFLASH_KERNEL_SIMT);
    size_t need = tree_attn_layout(p).total;
    if (tree_attn_kernel(dims, DFLASH_KERNEL_AUTO) == DFLASH_KERNEL_TC) {
        tree_attn_plan(p, DFLASH_KERNEL_TC);
        need = std::max(need, tree_attn_layout(p).total);
    }
    return need;
}

dflash_status dflash_tree_attn_err(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                                   const int32_t* seq_lens, const int32_t* parents, const int32_t* num_nodes,
                                   const dflash_dims* dims, int32_t max_nodes, int32_t window, float scale, void* out,
                                   float* lse, dflash_kernel kernel, uint32_t* device_error, void* workspace,
                                   size_t workspace_bytes, uint32_t wait_limit_us, void* stream)
{
    clear_error();
    const dflash_status s = check_attn_dims(dims, max_nodes, DFLASH_MAX_TREE_NODES, 1);
    if (s != DFLASH_OK) return s;
    if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !parents || !out)
        return report_error(DFLASH_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return report_error(DFLASH_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    if (out == q) return report_error(DFLASH_ERR_INVALID_ARG, "out must not alias q");
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(parents, 4) || !aligned(num_nodes, 4) ||
        !aligned(lse, 4) || !aligned(device_error, 4))
        return report_error(DFLASH_ERR_INVALID_ARG,
                            "page_table, seq_lens, parents, num_nodes, lse and device_error must be 4-byte aligned");
    if (window < 0) return report_error(DFLASH_ERR_INVALID_ARG, "window %d < 0", window);
    if (!std::isfinite(scale) || !(scale > 0.f))
        return report_error(DFLASH_ERR_INVALID_ARG, "scale must be finite and > 0");
    const int which = tree_attn_kernel(dims, (int32_t)kernel);
    if (which == -DFLASH_ERR_UNSUPPORTED)
        return report_error(DFLASH_ERR_UNSUPPORTED, "the tensor-core kernel takes bf16 caches of strides > 0");
    if (which < 0) return report_error(DFLASH_ERR_INVALID_ARG, "unknown kernel selector %d", (int)kernel);
    TreeAttnParams p{};
    fill_sizes(p, dims, max_nodes);
    tree_attn_plan(p, which);
    const TreeAttnLayout wl = tree_attn_layout(p);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < wl.total)
        return report_error(DFLASH_ERR_WORKSPACE, "tree attention needs a 256-byte aligned workspace of %zu bytes",
                            wl.total);
    char* wsb = static_cast<char*>(workspace);
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.parents = parents;
    p.num_nodes = num_nodes;
    p.out = out;
    p.lse = lse;
    p.err = device_error ? device_error : reinterpret_cast<uint32_t*>(wsb);
    p.part_lse = reinterpret_cast<float*>(wsb + wl.lse_off);
    p.part_out = reinterpret_cast<float*>(wsb + wl.out_off);
    p.window = window;
    p.scale = scale;
    p.wait_ns = wait_limit_us ? (unsigned long long)wait_limit_us * 1000ull : DFLASH_DEFAULT_WAIT_NS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = which == DFLASH_KERNEL_TC ? launch_tree_attn_tc(p, st) : launch_tree_attn_simt(p, st);
    if (e != cudaSuccess) return cuda_fail(e, "tree attention kernel launch");
    e = launch_tree_join(p, st);
    if (e != cudaSuccess) return cuda_fail(e, "tree attention join launch");
    return DFLASH_OK;
}

dflash_status dflash_tree_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                               const int32_t* seq_lens, const int32_t* parents, const int32_t* num_nodes,
                               const dflash_dims* dims, int32_t max_nodes, int32_t window, float scale, void* out,
                               float* lse, dflash_kernel kernel, void* workspace, size_t workspace_bytes,
                               uint32_t wait_limit_us, void* stream)
{
    return dflash_tree_attn_err(q, k_cache, v_cache, page_table, seq_lens, parents, num_nodes, dims, max_nodes, window,
                                scale, out, lse, kernel, nullptr, workspace, workspace_bytes, wait_limit_us, stream);
}

dflash_status dflash_shared_error_word(uint32_t** word)
{
    clear_error();
    if (!word) return report_error(DFLASH_ERR_INVALID_ARG, "NULL pointer");
    const cudaError_t e = shared_error_word(word);
    return e == cudaSuccess ? DFLASH_OK : cuda_fail(e, "address of the error word");
}

size_t dflash_logprobs_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t top_k)
{
    if (num_rows < 0 || num_rows > 65535 || vocab < 1) return 0;
    if (top_k < 0 || top_k > DFLASH_MAX_TOP_K || top_k > vocab) return 0;
    return logprobs_layout(num_rows, logprobs_slices(std::max(1, num_rows), vocab), top_k).total;
}

dflash_status dflash_token_logprobs(const void* logits, dflash_dtype dtype, int32_t num_rows, int32_t vocab,
                                    int64_t row_stride, float temperature, const int32_t* tokens, int32_t num_tokens,
                                    float* token_logp, float* log_z, float* entropy, int32_t top_k,
                                    int32_t* top_tokens, float* top_logp, uint32_t* device_error, void* workspace,
                                    size_t workspace_bytes, void* stream)
{
    clear_error();
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP32)
        return report_error(DFLASH_ERR_INVALID_ARG, "dtype must be bf16 or fp32");
    if (num_rows < 0 || num_rows > 65535)
        return report_error(DFLASH_ERR_INVALID_ARG, "num_rows %d outside [0, 65535]", num_rows);
    if (vocab < 1) return report_error(DFLASH_ERR_INVALID_ARG, "vocab %d < 1", vocab);
    if (row_stride < vocab)
        return report_error(DFLASH_ERR_INVALID_ARG, "row_stride %lld < vocab", (long long)row_stride);
    if (!std::isfinite(temperature) || !(temperature >= 1e-30f))
        return report_error(DFLASH_ERR_INVALID_ARG, "temperature must be finite and >= 1e-30");
    if (num_tokens < 0 || num_tokens > 64)
        return report_error(DFLASH_ERR_INVALID_ARG, "num_tokens %d outside [0, 64]", num_tokens);
    if (top_k < 0 || top_k > DFLASH_MAX_TOP_K || top_k > vocab)
        return report_error(DFLASH_ERR_INVALID_ARG, "top_k %d outside [0, min(vocab, %d)]", top_k, DFLASH_MAX_TOP_K);
    if (num_rows == 0) return DFLASH_OK;
    if (!logits || (num_tokens && (!tokens || !token_logp)) || (top_k && (!top_tokens || !top_logp)))
        return report_error(DFLASH_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(logits, dtype == DFLASH_BF16 ? 2 : 4) || !aligned(tokens, 4) || !aligned(token_logp, 4) ||
        !aligned(log_z, 4) || !aligned(entropy, 4) || !aligned(top_tokens, 4) || !aligned(top_logp, 4) ||
        !aligned(device_error, 4))
        return report_error(DFLASH_ERR_INVALID_ARG,
                            "misaligned pointer (logits to their element size, the rest 4 bytes)");
    LogprobsParams p{};
    p.slices = logprobs_slices(num_rows, vocab);
    const LogprobsLayout wl = logprobs_layout(num_rows, p.slices, top_k);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < wl.total)
        return report_error(DFLASH_ERR_WORKSPACE, "log probabilities need a 256-byte aligned workspace of %zu bytes",
                            wl.total);
    char* wsb = static_cast<char*>(workspace);
    p.logits = logits;
    p.dtype = dtype;
    p.R = num_rows;
    p.V = vocab;
    p.row_stride = row_stride;
    p.temperature = temperature;
    p.tokens = tokens;
    p.m = num_tokens;
    p.token_logp = token_logp;
    p.log_z = log_z;
    p.entropy = entropy;
    p.k = top_k;
    p.top_tokens = top_tokens;
    p.top_logp = top_logp;
    p.err = device_error;
    p.counters = reinterpret_cast<int32_t*>(wsb);
    p.part_stat = reinterpret_cast<float*>(wsb + wl.stat_off);
    p.part_key = reinterpret_cast<unsigned long long*>(wsb + wl.key_off);
    const cudaError_t e = launch_token_logprobs(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "log probability kernel launch");
    return DFLASH_OK;
}

size_t dflash_tree_accept_workspace_bytes(void) { return 2 * kKeyBytes; }

dflash_status dflash_tree_accept(const void* logits, dflash_dtype dtype, int32_t batch, int32_t max_nodes,
                                 int32_t vocab, int64_t row_stride, const int32_t* tokens, const int32_t* parents,
                                 const int32_t* num_nodes, int32_t* accepted_len, int32_t* path, int32_t* next_token,
                                 int32_t* target_argmax, uint32_t* device_error, void* workspace,
                                 size_t workspace_bytes, void* stream)
{
    clear_error();
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP32)
        return report_error(DFLASH_ERR_INVALID_ARG, "dtype must be bf16 or fp32");
    if (max_nodes < 1 || max_nodes > DFLASH_MAX_TREE_NODES)
        return report_error(DFLASH_ERR_INVALID_ARG, "max_nodes %d outside [1, %d]", max_nodes, DFLASH_MAX_TREE_NODES);
    if (batch < 1 || (int64_t)batch * max_nodes > 65535)
        return report_error(DFLASH_ERR_INVALID_ARG, "batch %d x max_nodes %d outside [1, 65535]", batch, max_nodes);
    if (vocab < 1) return report_error(DFLASH_ERR_INVALID_ARG, "vocab %d < 1", vocab);
    if (row_stride < vocab)
        return report_error(DFLASH_ERR_INVALID_ARG, "row_stride %lld < vocab", (long long)row_stride);
    if (!logits || !tokens || !parents || !accepted_len || !path || !next_token)
        return report_error(DFLASH_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(logits, dtype == DFLASH_BF16 ? 2 : 4) || !aligned(tokens, 4) || !aligned(parents, 4) ||
        !aligned(num_nodes, 4) || !aligned(accepted_len, 4) || !aligned(path, 4) || !aligned(next_token, 4) ||
        !aligned(target_argmax, 4) || !aligned(device_error, 4))
        return report_error(DFLASH_ERR_INVALID_ARG,
                            "misaligned pointer (logits to their element size, the rest 4 bytes)");
    const size_t need = dflash_tree_accept_workspace_bytes();
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
        return report_error(DFLASH_ERR_WORKSPACE, "tree acceptance needs a 256-byte aligned workspace of %zu bytes",
                            need);
    TreeAcceptParams p{};
    p.logits = logits;
    p.dtype = dtype;
    p.B = batch;
    p.T = max_nodes;
    p.V = vocab;
    p.row_stride = row_stride;
    p.tokens = tokens;
    p.parents = parents;
    p.num_nodes = num_nodes;
    p.accepted = accepted_len;
    p.path = path;
    p.next_token = next_token;
    p.target_argmax = target_argmax;
    p.err = device_error;
    p.keys = static_cast<unsigned long long*>(workspace);
    p.counters = p.keys + kKeyBytes / sizeof(unsigned long long);
    const cudaError_t e = launch_tree_accept(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tree acceptance kernel launch");
    return DFLASH_OK;
}

dflash_status dflash_tree_commit(void* k_cache, void* v_cache, const int32_t* page_table, const int32_t* seq_lens,
                                 const int32_t* path, const int32_t* accepted_len, const int32_t* num_nodes,
                                 int32_t* new_lens, const dflash_dims* dims, int32_t max_nodes, int32_t num_layers,
                                 int64_t layer_stride, uint32_t* device_error, void* stream)
{
    clear_error();
    const dflash_status s = check_attn_dims(dims, max_nodes, DFLASH_MAX_TREE_NODES, 1);
    if (s != DFLASH_OK) return s;
    const int64_t es = dims->dtype == DFLASH_BF16 ? 2 : 4;
    if (num_layers < 1 || num_layers > 65535)
        return report_error(DFLASH_ERR_INVALID_ARG, "num_layers %d outside [1, 65535]", num_layers);
    if (num_layers > 1 && (layer_stride <= 0 || (layer_stride * es) % 16))
        return report_error(DFLASH_ERR_INVALID_ARG, "layer_stride must be positive and a multiple of 16 bytes");
    if (dims->kv_stride_slot <= 0 || (dims->num_pages > 1 && dims->kv_stride_page <= 0))
        return report_error(DFLASH_ERR_INVALID_ARG, "slots and pages of a cache that is written need strides > 0");
    if (!k_cache || !v_cache || !page_table || !seq_lens || !path || !accepted_len)
        return report_error(DFLASH_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(path, 4) || !aligned(accepted_len, 4) || !aligned(num_nodes, 4) || !aligned(new_lens, 4) ||
        !aligned(device_error, 4))
        return report_error(DFLASH_ERR_INVALID_ARG, "misaligned pointer (caches 16 bytes, the rest 4)");
    if (k_cache == v_cache) return report_error(DFLASH_ERR_INVALID_ARG, "k_cache and v_cache must not be one cache");
    const char* nl = reinterpret_cast<const char*>(new_lens);
    const size_t lens_bytes = sizeof(int32_t) * (size_t)dims->batch;
    auto overlaps = [&](const void* a, size_t bytes) {
        const char* c = static_cast<const char*>(a);
        return nl && c && nl < c + bytes && c < nl + lens_bytes;
    };
    if ((new_lens != seq_lens && overlaps(seq_lens, lens_bytes)) || overlaps(accepted_len, lens_bytes) ||
        overlaps(num_nodes, lens_bytes) || overlaps(path, lens_bytes * max_nodes) ||
        overlaps(page_table, lens_bytes * dims->max_pages))
        return report_error(DFLASH_ERR_INVALID_ARG, "new_lens may be seq_lens itself but overlap no other input");
    TreeCommitParams p{};
    p.k = k_cache;
    p.v = v_cache;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.path = path;
    p.accepted = accepted_len;
    p.num_nodes = num_nodes;
    p.new_lens = new_lens;
    p.err = device_error;
    p.B = dims->batch;
    p.T = max_nodes;
    p.layers = num_layers;
    p.Hkv = dims->num_kv_heads;
    p.row_bytes = (int32_t)(dims->head_dim * es);
    p.page_size = dims->page_size;
    p.num_pages = dims->num_pages;
    p.max_pages = dims->max_pages;
    p.max_seq_len = max_len_of(dims);
    p.sp = dims->kv_stride_page * es;
    p.ss = dims->kv_stride_slot * es;
    p.sh = dims->kv_stride_head * es;
    p.sl = num_layers > 1 ? layer_stride * es : 0;
    const cudaError_t e = launch_tree_commit(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tree commit kernel launch");
    return DFLASH_OK;
}

}  // extern "C"
