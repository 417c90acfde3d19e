// Join of the tree attention's partials: a (request, KV head) pair whose key tiles lie in several
// ranges has one normalised partial (o_c, lse_c) per range and row, and
//   m = max_c lse_c, w_c = exp(lse_c - m), out = sum_c w_c o_c / sum_c w_c, lse = m + log(sum_c w_c).
// A partial of scores that are not finite has a NaN lse; the maximum hands it on, so that the row is NaN as a whole
// pair's would be. Pairs that one range holds whole are final already. A request with a bad length or tree size gets
// its zeros here.
//
// A warp takes a row, or where there are few rows 2, 4 or 8 warps take one, a stretch of its partials each, and add
// theirs up in shared memory, in order. A warp's lanes read the partials' lse values (32 at a time) and form the weights
// while the first partial rows come, four to sixteen a time. Launched as a programmatic dependent of the attention
// kernel; the deal of tiles to ranges is worked out before the wait for it. Bound: trips to L2, two to start with and
// one more per batch of partials; behind the attention it adds 3 to 7 us. Measured, whole calls of one request after a
// flush of L2: 1 node, 16/1 heads of 128, 100k keys (151 partials a row) 33 us, 51 with a warp per row; 7 nodes, 12/2
// heads of 96, 18k keys 22.5, 41 with a warp per row (back to back on inputs beyond L2 25 and 17 now).
//
// Every CTA walks all requests twice, 32 a step, to find its ranges, so that the time of large batches grows with
// their square: 4 nodes, 200 to 300 keys, 32/8 heads of 128, 256 requests 127 us, 1024 573, 4096 4660.
#include <algorithm>
#include <cmath>

#include "tree_attn.cuh"

namespace dflash {
namespace {

__device__ __align__(256) uint32_t g_error_block[(256 + DFLASH_COUNTER_BYTES) / sizeof(uint32_t)];

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Partials whose loads a warp has in flight, of V floats a lane, and the CTAs that an SM then holds.
template <int V>
constexpr int kAheadOf = V == 2 ? 16 : V == 8 ? 8 : 4;
template <int V>
constexpr int kCtasOf = V == 4 ? 4 : 2;

template <int V, bool kShare>  // floats per lane: DV <= 32 V; several warps to a row
__global__ void __launch_bounds__(kThreads, kCtasOf<V>)
    tree_join_kernel(const TreeAttnParams p, const int32_t warps_a_row)
{
    __shared__ int32_t sh_r0, sh_parts;
    __shared__ float sh_acc[kShare ? kWarps : 1][V][32], sh_m[kWarps], sh_t[kWarps];
    const int32_t pair = blockIdx.x;
    const int32_t b = pair / p.Hkv, g = pair % p.Hkv;
    const int32_t sub = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SubTile st = sub_tile(p, sub);
    const TreeReq rq = tree_request(p, b);
    const int32_t node0 = st.rt * p.npt;
    if (rq.bad && g == 0 && sub == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        raise_error(p.err, tree_request_error(p, rq));
    const int32_t n_here = rq.bad ? p.T : rq.n;
    const int32_t live = min(p.npt, n_here - node0) * p.Gc;
    int32_t r0 = 0, parts = 0;
    if (rq.nt > 0 && live > 0) {
        if (warp == 0) {
            const int64_t first = tree_weight_before(p, b) + g * tree_weight(p, rq), total = tree_weight_before(p, p.B);
            const int32_t used = ranges_used(p, total);
            if (lane == 0) {
                sh_r0 = range_of(total, used, first + p.pair_cost);  // its tiles follow its fixed cost
                sh_parts = range_of(total, used, first + tree_weight(p, rq) - 1) - sh_r0 + 1;
            }
        }
        __syncthreads();
        r0 = sh_r0;
        parts = sh_parts;
    }
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();  // the next layer's attention may set itself up; it waits for this grid
    if (live <= 0 || parts == 1 || (parts == 0 && !rq.bad)) return;
    const int32_t d_here = min(p.DV, p.D - st.dv * p.DV);
    // A lane's floats: runs of four (two, of 64 dims), 128 dims apart, so that a warp's loads are whole lines.
    constexpr int kRun = V < 4 ? 2 : 4;
    const int32_t d0 = lane * kRun;
    auto dim_of = [&](int u) -> int32_t { return d0 + u / kRun * 128; };  // of run u / kRun
    const int32_t share = kShare ? warps_a_row : 1;
    // `share` warps to a row: this one's partials are [c0, c1). No fewer than it loads at once, so that few partials
    // are one warp's.
    constexpr int kAhead = kAheadOf<V>;
    const int32_t member = warp % share, rows_here = kWarps / share, per = kShare ? max(kAhead, (parts + share - 1) / share) : parts;
    const int32_t c0 = min(parts, member * per), c1 = min(parts, c0 + per);
    const int32_t one = min(c1 - c0, 32);
    for (int32_t row0 = blockIdx.z * rows_here; row0 < live; row0 += gridDim.z * rows_here) {
        const int32_t row = row0 + warp / share;
        if (!kShare && row >= live) break;
        const bool on_row = !kShare || row < live;
        // part c's row: the pair's first part is in slot 1 of its range, the others in slot 0
        auto part_at = [&](int32_t c) -> int64_t { return tree_part_row(p, r0 + c, sub, c == 0 ? 1 : 0) + row; };
        auto load = [&](int32_t c, bool live_part, float (&x)[V]) {
            const float* src = p.part_out + part_at(live_part ? c : c0) * p.DV;
#pragma unroll
            for (int u = 0; u < V; u += kRun) {
                const bool on = live_part && dim_of(u) < d_here;
                if (V < 4) {
                    const float2 y = on ? __ldcg(reinterpret_cast<const float2*>(src + dim_of(u)))
                                        : make_float2(0.f, 0.f);
                    x[u] = y.x;
                    x[u + 1] = y.y;
                } else {
                    const float4 y = on ? __ldcg(reinterpret_cast<const float4*>(src + dim_of(u)))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[u] = y.x;
                    x[u + 1] = y.y;
                    x[(u + 2) % V] = y.z;
                    x[(u + 3) % V] = y.w;
                }
            }
        };
        // The first parts' values are on their way beside the lse values that weigh them: one trip to L2, mostly.
        float lse0 = -INFINITY, ahead[kAhead][V];
        float m = -INFINITY, t = 0.f, acc[V];
#pragma unroll
        for (int u = 0; u < V; ++u) acc[u] = 0.f;
        if (on_row && c0 < c1) {
            lse0 = lane < one ? __ldcg(p.part_lse + part_at(c0 + lane)) : -INFINITY;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load(c0 + k, c0 + k < c1, ahead[k]);
            m = lse0;
            for (int32_t c = c0 + 32 + lane; c < c1; c += 32) m = max_nan(m, __ldcg(p.part_lse + part_at(c)));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        }
        if (m != -INFINITY) {
            // (a partial without a visible key is 0 and so is its weight)
            float w = lse0 == -INFINITY ? 0.f : expf(lse0 - m);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);  // 0 past the parts
                t += wk;
#pragma unroll
                for (int u = 0; u < V; ++u) acc[u] = fmaf(wk, ahead[k][u], acc[u]);
            }
            for (int32_t at = kAhead; c0 + at < c1; at += kAhead) {
                if (at % 32 == 0) {
                    const int32_t c = c0 + at + lane;
                    const float l = c < c1 ? __ldcg(p.part_lse + part_at(c)) : -INFINITY;
                    w = l == -INFINITY ? 0.f : expf(l - m);
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) load(c0 + at + k, c0 + at + k < c1, ahead[k]);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, (at + k) & 31);
                    t += wk;
#pragma unroll
                    for (int u = 0; u < V; ++u) acc[u] = fmaf(wk, ahead[k][u], acc[u]);
                }
            }
        }
        if (kShare && per < parts) {
#pragma unroll
            for (int u = 0; u < V; ++u) sh_acc[warp][u][lane] = acc[u];
            if (lane == 0) {
                sh_m[warp] = m;
                sh_t[warp] = t;
            }
            __syncthreads();
            if (member == 0) {
                for (int i = 1; i < share; ++i) m = max_nan(m, sh_m[warp + i]);
                t = 0.f;
#pragma unroll
                for (int u = 0; u < V; ++u) acc[u] = 0.f;
                for (int i = 0; i < share; ++i) {
                    const float mi = sh_m[warp + i], wi = mi == -INFINITY ? 0.f : expf(mi - m);
                    t = fmaf(wi, sh_t[warp + i], t);
#pragma unroll
                    for (int u = 0; u < V; ++u) acc[u] = fmaf(wi, sh_acc[warp + i][u][lane], acc[u]);
                }
            }
            __syncthreads();
        }
        if (member != 0 || !on_row) continue;
        const float inv = tree_inv_sum(t, !rq.bad);
        const int32_t node = node0 + row / p.Gc, head = g * p.G + st.gc * p.Gc + row % p.Gc;
        const int64_t orow = ((int64_t)b * p.T + node) * p.Hq + head;
#pragma unroll
        for (int u = 0; u < V; u += 2) {
            const int32_t d = dim_of(u) + u % kRun;
            if (d >= d_here) continue;
            const int64_t o = orow * p.D + st.dv * p.DV + d;
            if (p.dtype == DFLASH_BF16)
                *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + o) =
                    __floats2bfloat162_rn(acc[u] * inv, acc[u + 1] * inv);
            else
                *reinterpret_cast<float2*>(static_cast<float*>(p.out) + o) =
                    make_float2(acc[u] * inv, acc[u + 1] * inv);
        }
        if (lane == 0 && st.dv == 0 && p.lse) p.lse[orow] = tree_row_lse(m + logf(t), t, !rq.bad);
    }
}

}  // namespace

template <int V>
static cudaError_t launch_join(const TreeAttnParams& p, cudaStream_t stream)
{
    // about one wave of warps: a warp takes several rows of a large call, several warps take one of a small one
    const int64_t wave = (int64_t)device_sm_count() * kCtasOf<V>, tiles = (int64_t)p.B * p.Hkv * p.n_sub;
    int32_t share = 1;
    while (share < kWarps && tiles * p.rows * share * 2 <= wave * kWarps) share *= 2;
    const int64_t most = (p.rows * share + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv), (unsigned)p.n_sub,
                       (unsigned)std::max<int64_t>(1, std::min(most, (wave + tiles - 1) / tiles)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return share > 1 ? cudaLaunchKernelEx(&cfg, tree_join_kernel<V, true>, p, share)
                     : cudaLaunchKernelEx(&cfg, tree_join_kernel<V, false>, p, share);
}

cudaError_t shared_error_word(uint32_t** word)
{
    void* at = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&at, g_error_block);
    if (e == cudaSuccess) *word = static_cast<uint32_t*>(at);
    return e;
}

cudaError_t launch_tree_join(const TreeAttnParams& p, cudaStream_t stream)
{
    // a lane's floats: the narrowest that cover the partial's row (DV is a multiple of 16)
    if (p.DV <= 64) return launch_join<2>(p, stream);
    if (p.DV <= 128) return launch_join<4>(p, stream);
    if (p.DV <= 256) return launch_join<8>(p, stream);
    return launch_join<16>(p, stream);
}

}  // namespace dflash
