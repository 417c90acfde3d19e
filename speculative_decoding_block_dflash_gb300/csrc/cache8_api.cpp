// C-ABI front end of the rotary positions and the 8-bit cache: host-side validation, plans, workspace carve-up and
// launches. See include/dflash_attn.h for the contract of each entry point.
#include <algorithm>
#include <cmath>

#include "cache8.h"

namespace dflash {
namespace {

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
void clear_error() { report_error(DFLASH_OK, "%s", ""); }
int32_t elem(int32_t dtype) { return dtype == DFLASH_BF16 ? 2 : 4; }

dflash_status check_rope(const dflash_rope_freqs* r, int32_t D)
{
    if (!r->turns || !aligned(r->turns, 8))
        return report_error(DFLASH_ERR_INVALID_ARG, "the table of frequencies is NULL or not 8-byte aligned");
    if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > D)
        return report_error(DFLASH_ERR_INVALID_ARG, "rotary_dim %d must be even, in [2, head_dim = %d]", r->rotary_dim, D);
    if (r->layout != DFLASH_ROPE_HALF && r->layout != DFLASH_ROPE_INTERLEAVED)
        return report_error(DFLASH_ERR_INVALID_ARG, "unknown rotary layout %d", r->layout);
    if (!std::isfinite(r->gain) || !(r->gain > 0.f))
        return report_error(DFLASH_ERR_INVALID_ARG, "the gain must be finite and > 0");
    return DFLASH_OK;
}

// Rows [N, H, D] whose units are whole and 16-byte aligned.
bool vector_rows(const void* p, int64_t st, int64_t sh, int32_t dtype, int32_t D, int32_t half)
{
    const int32_t n = 16 / elem(dtype);
    return aligned(p, 16) && st % n == 0 && sh % n == 0 && D % 16 == 0 && half % 8 == 0;
}

dflash_status check_rows(const char* what, const void* p, int64_t st, int64_t sh, int32_t dtype)
{
    if (!p) return report_error(DFLASH_ERR_INVALID_ARG, "%s is NULL", what);
    if (!aligned(p, elem(dtype))) return report_error(DFLASH_ERR_INVALID_ARG, "%s is not aligned to its elements", what);
    // (a stride of 0 repeats rows or heads)
    if (st < 0 || sh < 0) return report_error(DFLASH_ERR_INVALID_ARG, "negative stride of %s", what);
    return DFLASH_OK;
}

// The kernel that a call runs, or a negative status.
int attn_kernel(const dflash_dims* d, int32_t requested)
{
    if (requested == DFLASH_KERNEL_SIMT) return DFLASH_KERNEL_SIMT;
    if (requested != DFLASH_KERNEL_AUTO && requested != DFLASH_KERNEL_TC) return -DFLASH_ERR_INVALID_ARG;
    if (cache8_tc_supports(d)) return DFLASH_KERNEL_TC;
    return requested == DFLASH_KERNEL_TC ? -DFLASH_ERR_UNSUPPORTED : DFLASH_KERNEL_SIMT;
}

dflash_status check_attn8_dims(const dflash_dims* d, int32_t T)
{
    if (const dflash_status s = check_attn_dims(d, T, DFLASH_MAX_TREE_NODES, 1)) return s;
    if (d->kv_stride_page % 16 || d->kv_stride_slot % 16 || d->kv_stride_head % 16)
        return report_error(DFLASH_ERR_INVALID_ARG, "K/V strides must be multiples of 16 bytes");
    return DFLASH_OK;
}

}  // namespace

// Tree attention's plan on the CUDA cores. On the tensor cores few rows run on the kernel whose MMAs cost what the rows do
// (cache8_attn_few.cu), more in tiles of 128 on the other. Up to 32 rows: 8 requests of 2k to 16k keys, 32/8 heads of 128, took
// 59 us there with 8 queries (32 rows) against 61, 77 against 62 with 9, 103 against 65 with 16; one query of 32 such requests of
// 1k to 32k keys 196 against 319. Above 256 dims everything runs there, in tiles of up to 80 rows, as a CTA's TMEM holds their whole output.
void cache8_attn_plan(TreeAttnParams& p, int kernel)
{
    if (kernel != DFLASH_KERNEL_TC) {
        tree_attn_plan(p, kernel);
        return;
    }
    const int32_t rows = p.T * p.G;
    p.few = rows <= 32 || p.D > 256;
    const int32_t most = p.few ? 80 : 128;
    p.Gc = 1;
    for (int32_t gc = std::min(p.G, most); gc >= 1; --gc)
        if (p.G % gc == 0) {
            p.Gc = gc;
            break;
        }
    const int32_t fit = most / p.Gc;
    p.nrt = (p.T + fit - 1) / fit;
    p.npt = (p.T + p.nrt - 1) / p.nrt;  // query tiles of equal size
    p.rows = p.npt * p.Gc;
    p.tile = 128;
    p.pair = 0;
    p.pair_cost = p.few ? 4 : 8;  // a piece's fixed cost, in tiles
    p.DV = p.few ? p.D : p.D <= 64 ? 64 : p.D <= 128 ? 128 : 256;
    p.ndv = 1;
    p.n_sub = (p.G / p.Gc) * p.nrt;
    p.ranges = std::max(1, device_sm_count() / p.n_sub);  // one wave of one CTA per SM
}

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_rope(const void* x, void* out, dflash_dtype dtype, int32_t num_tokens, int32_t num_heads,
                          int32_t head_dim, int64_t x_stride_token, int64_t x_stride_head, int64_t out_stride_token,
                          int64_t out_stride_head, const int32_t* positions, const dflash_rope_freqs* freqs,
                          int32_t inverse, void* stream)
{
    clear_error();
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP32)
        return report_error(DFLASH_ERR_INVALID_ARG, "dtype must be bf16 or fp32");
    if (num_tokens < 0 || num_tokens > DFLASH_PROJECT_MAX_TOKENS)
        return report_error(DFLASH_ERR_INVALID_ARG, "num_tokens %d outside [0, %d]", num_tokens,
                            DFLASH_PROJECT_MAX_TOKENS);
    if (num_heads < 1 || num_heads > 1024)
        return report_error(DFLASH_ERR_INVALID_ARG, "num_heads %d outside [1, 1024]", num_heads);
    if (head_dim < 2 || head_dim > DFLASH_MAX_HEAD_DIM)
        return report_error(DFLASH_ERR_INVALID_ARG, "head_dim %d outside [2, %d]", head_dim, DFLASH_MAX_HEAD_DIM);
    if (inverse != 0 && inverse != 1) return report_error(DFLASH_ERR_INVALID_ARG, "inverse must be 0 or 1");
    if (!freqs) return report_error(DFLASH_ERR_INVALID_ARG, "freqs is NULL");
    if (const dflash_status s = check_rope(freqs, head_dim)) return s;
    if (num_tokens == 0) return DFLASH_OK;
    if (const dflash_status s = check_rows("x", x, x_stride_token, x_stride_head, dtype)) return s;
    if (const dflash_status s = check_rows("out", out, out_stride_token, out_stride_head, dtype)) return s;
    // the rows one behind the other at the smaller stride, and those at the larger behind them
    const bool heads_inside = out_stride_head <= out_stride_token;
    const int64_t near = heads_inside ? out_stride_head : out_stride_token, far = heads_inside ? out_stride_token : out_stride_head;
    const int64_t near_n = heads_inside ? num_heads : num_tokens;
    if ((num_heads > 1 && out_stride_head < head_dim) || (num_tokens > 1 && out_stride_token < head_dim) ||
        (num_heads > 1 && num_tokens > 1 && far < (near_n - 1) * near + head_dim))
        return report_error(DFLASH_ERR_INVALID_ARG, "the strides of out (%lld, %lld) let its rows overlap",
                            (long long)out_stride_token, (long long)out_stride_head);
    if (!positions || !aligned(positions, 4))
        return report_error(DFLASH_ERR_INVALID_ARG, "positions is NULL or not 4-byte aligned");
    const bool same = (num_tokens == 1 || x_stride_token == out_stride_token) &&
                      (num_heads == 1 || x_stride_head == out_stride_head);
    if (x == out && !same) return report_error(DFLASH_ERR_INVALID_ARG, "in place, x and out must have the same strides");
    RopeParams p{};
    p.x = x;
    p.out = out;
    p.positions = positions;
    p.turns = freqs->turns;
    p.dtype = dtype;
    p.N = num_tokens;
    p.H = num_heads;
    p.D = head_dim;
    p.half = freqs->rotary_dim / 2;
    p.interleaved = freqs->layout == DFLASH_ROPE_INTERLEAVED;
    p.xt = x_stride_token;
    p.xh = x_stride_head;
    p.ot = out_stride_token;
    p.oh = out_stride_head;
    p.gain = freqs->gain;
    p.inverse = inverse;
    p.vec = vector_rows(x, p.xt, p.xh, dtype, p.D, p.half) && vector_rows(out, p.ot, p.oh, dtype, p.D, p.half);
    p.in_place = x == out;
    const cudaError_t e = launch_rope(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DFLASH_OK
                            : report_error(DFLASH_ERR_CUDA, "rotary kernel launch: %s", cudaGetErrorString(e));
}

dflash_status dflash_append_kv(const void* k, const void* v, int32_t num_tokens, int64_t k_stride_token,
                               int64_t k_stride_head, int64_t v_stride_token, int64_t v_stride_head,
                               const int32_t* starts, const int32_t* positions, const dflash_rope_freqs* freqs,
                               void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int32_t* page_table,
                               const int32_t* seq_lens, const dflash_dims* dims, uint32_t* device_error, void* stream)
{
    clear_error();
    if (const dflash_status s = check_attn_dims(dims, 1, 1, 1)) return s;
    if (num_tokens < 0 || num_tokens > DFLASH_PROJECT_MAX_TOKENS)
        return report_error(DFLASH_ERR_INVALID_ARG, "num_tokens %d outside [0, %d]", num_tokens,
                            DFLASH_PROJECT_MAX_TOKENS);
    if (!k_scale != !v_scale) return report_error(DFLASH_ERR_INVALID_ARG, "give both scales (e4m3 caches) or none");
    if (k_scale && (dims->kv_stride_page % 16 || dims->kv_stride_slot % 16 || dims->kv_stride_head % 16))
        return report_error(DFLASH_ERR_INVALID_ARG, "K/V strides must be multiples of 16 bytes");
    if (freqs)
        if (const dflash_status s = check_rope(freqs, dims->head_dim)) return s;
    if (!k_cache || !v_cache || !page_table || !seq_lens) return report_error(DFLASH_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
        return report_error(DFLASH_ERR_INVALID_ARG, "k_cache and v_cache must be 16-byte aligned");
    if (k_cache == v_cache) return report_error(DFLASH_ERR_INVALID_ARG, "k_cache and v_cache must not be the same");
    if (k_scale && k_scale == v_scale) return report_error(DFLASH_ERR_INVALID_ARG, "k_scale and v_scale must not be the same");
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(starts, 4) || !aligned(positions, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(device_error, 4))
        return report_error(DFLASH_ERR_INVALID_ARG, "page_table, seq_lens, starts, positions, the scales and device_error "
                                                    "must be 4-byte aligned");
    if (!starts && num_tokens % dims->batch)
        return report_error(DFLASH_ERR_INVALID_ARG, "%d tokens without starts are not a multiple of the batch %d",
                            num_tokens, dims->batch);
    if (num_tokens == 0) return DFLASH_OK;
    if (const dflash_status s = check_rows("k", k, k_stride_token, k_stride_head, dims->dtype)) return s;
    if (const dflash_status s = check_rows("v", v, v_stride_token, v_stride_head, dims->dtype)) return s;
    AppendParams p{};
    p.k = k;
    p.v = v;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.starts = starts;
    p.positions = positions;
    p.err = device_error;
    p.dtype = dims->dtype;
    p.N = num_tokens;
    p.B = dims->batch;
    p.Hkv = dims->num_kv_heads;
    p.D = dims->head_dim;
    if (freqs) {
        p.turns = freqs->turns;
        p.half = freqs->rotary_dim / 2;
        p.interleaved = freqs->layout == DFLASH_ROPE_INTERLEAVED;
        p.gain = freqs->gain;
    }
    p.kt = k_stride_token;
    p.kh = k_stride_head;
    p.vt = v_stride_token;
    p.vh = v_stride_head;
    p.page_size = dims->page_size;
    p.num_pages = dims->num_pages;
    p.max_pages = dims->max_pages;
    p.max_seq_len = dims->max_seq_len ? dims->max_seq_len : dims->max_pages * dims->page_size;
    p.sp = dims->kv_stride_page;
    p.ss = dims->kv_stride_slot;
    p.sh = dims->kv_stride_head;
    p.vec_k = vector_rows(k, p.kt, p.kh, p.dtype, p.D, p.half);
    p.vec_v = vector_rows(v, p.vt, p.vh, p.dtype, p.D, 0);
    const cudaError_t e = launch_append_kv(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DFLASH_OK
                            : report_error(DFLASH_ERR_CUDA, "append kernel launch: %s", cudaGetErrorString(e));
}

size_t dflash_cache8_attn_workspace_bytes(const dflash_dims* dims, int32_t max_queries)
{
    clear_error();
    if (check_attn8_dims(dims, max_queries) != DFLASH_OK) return 0;
    TreeAttnParams p{};
    tree_fill_sizes(p, dims, max_queries);
    cache8_attn_plan(p, DFLASH_KERNEL_SIMT);
    size_t need = tree_attn_layout(p).total;
    if (attn_kernel(dims, DFLASH_KERNEL_AUTO) == DFLASH_KERNEL_TC) {
        cache8_attn_plan(p, DFLASH_KERNEL_TC);
        need = std::max(need, tree_attn_layout(p).total);
    }
    return need;
}

dflash_status dflash_cache8_attn(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                 const float* v_scale, const int32_t* page_table, const int32_t* seq_lens,
                                 const int32_t* num_queries, const int32_t* parents, const dflash_dims* dims,
                                 int32_t max_queries, int32_t causal, int32_t window, float scale, void* out, float* lse,
                                 dflash_kernel kernel, uint32_t* device_error, void* workspace, size_t workspace_bytes,
                                 uint32_t wait_limit_us, void* stream)
{
    clear_error();
    if (const dflash_status s = check_attn8_dims(dims, max_queries)) return s;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !page_table || !seq_lens || !out)
        return report_error(DFLASH_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return report_error(DFLASH_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    if (out == q) return report_error(DFLASH_ERR_INVALID_ARG, "out must not alias q");
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(parents, 4) || !aligned(num_queries, 4) || !aligned(lse, 4) || !aligned(device_error, 4))
        return report_error(DFLASH_ERR_INVALID_ARG, "the scales, page_table, seq_lens, parents, num_queries, lse and "
                                                    "device_error must be 4-byte aligned");
    if (causal != 0 && causal != 1) return report_error(DFLASH_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (parents && causal) return report_error(DFLASH_ERR_INVALID_ARG, "a tree has its own mask: causal must be 0");
    if (window < 0) return report_error(DFLASH_ERR_INVALID_ARG, "window %d < 0", window);
    if (!parents && !causal && window > 0 && window < max_queries)
        return report_error(DFLASH_ERR_INVALID_ARG, "window %d < max_queries %d of a non-causal block", window, max_queries);
    if (!std::isfinite(scale) || !(scale > 0.f))
        return report_error(DFLASH_ERR_INVALID_ARG, "scale must be finite and > 0");
    const int which = attn_kernel(dims, (int32_t)kernel);
    if (which == -DFLASH_ERR_UNSUPPORTED)
        return report_error(DFLASH_ERR_UNSUPPORTED, "the tensor-core kernel takes bf16 queries and caches of strides > 0");
    if (which < 0) return report_error(DFLASH_ERR_INVALID_ARG, "unknown kernel selector %d", (int)kernel);
    TreeAttnParams p{};
    tree_fill_sizes(p, dims, max_queries);
    cache8_attn_plan(p, which);
    const TreeAttnLayout wl = tree_attn_layout(p);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < wl.total)
        return report_error(DFLASH_ERR_WORKSPACE, "attention needs a 256-byte aligned workspace of %zu bytes", wl.total);
    char* wsb = static_cast<char*>(workspace);
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.parents = parents;
    p.num_nodes = num_queries;
    p.mask = parents ? kMaskTree : causal ? kMaskCausal : kMaskFull;
    p.out = out;
    p.lse = lse;
    p.err = device_error ? device_error : reinterpret_cast<uint32_t*>(wsb);
    p.part_lse = reinterpret_cast<float*>(wsb + wl.lse_off);
    p.part_out = reinterpret_cast<float*>(wsb + wl.out_off);
    p.window = window;
    p.scale = scale;
    p.wait_ns = wait_limit_us ? (unsigned long long)wait_limit_us * 1000ull : DFLASH_DEFAULT_WAIT_NS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = which == DFLASH_KERNEL_TC ? launch_cache8_attn_tc(p, st) : launch_cache8_attn_simt(p, st);
    if (e == cudaSuccess) e = launch_tree_join(p, st);
    return e == cudaSuccess ? DFLASH_OK
                            : report_error(DFLASH_ERR_CUDA, "attention kernel launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
