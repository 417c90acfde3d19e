// Join of the tree attention's partials: a (request, KV head) pair whose key tiles lie in several
// ranges has one normalised partial (o_c, lse_c) per range and row, and
//   m = max_c lse_c, w_c = exp(lse_c - m), out = sum_c w_c o_c / sum_c w_c, lse = m + log(sum_c w_c).
// Pairs that one range holds whole are final already. A request with a bad length or tree size gets its
// zeros here.
//
// A warp takes a row: its lanes read the partials' lse values (32 at a time) and form the weights while the first
// partial rows come, four to sixteen a time (2 requests of 2000 keys, 12 nodes of 8/2 heads, D = 64: 36 parts a row, 9.4
// us by itself with sixteen, 13.3 with four). Launched as a programmatic dependent of the attention kernel; the deal
// of tiles to ranges is worked out before the wait for it. Bound: trips to L2, two to start with and one more per batch
// of partials; behind the attention it adds 4 to 7 us.
#include <algorithm>
#include <cmath>

#include "tree_attn.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int V>  // floats per lane: DV <= 32 V
__global__ void __launch_bounds__(kThreads) tree_join_kernel(const TreeAttnParams p)
{
    __shared__ int32_t sh_r0, sh_parts;
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
            const int64_t first = tree_weight_before(p, b) + g * tree_weight(rq), total = tree_weight_before(p, p.B);
            const int32_t used = ranges_used(p, total);
            if (lane == 0) {
                sh_r0 = range_of(total, used, first + kPairCost);  // its tiles follow its fixed cost
                sh_parts = range_of(total, used, first + tree_weight(rq) - 1) - sh_r0 + 1;
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
    const int32_t one = min(parts, 32);
    for (int32_t row = blockIdx.z * kWarps + warp; row < live; row += gridDim.z * kWarps) {
        // part c's row: the pair's first part is in slot 1 of its range, the others in slot 0
        auto part_at = [&](int32_t c) -> int64_t { return tree_part_row(p, r0 + c, sub, c == 0 ? 1 : 0) + row; };
        auto load = [&](int32_t c, bool live_part, float (&x)[V]) {
            const float* src = p.part_out + part_at(live_part ? c : 0) * p.DV;
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
        constexpr int kAhead = V == 2 ? 16 : V == 8 ? 8 : 4;
        float lse0 = -INFINITY, ahead[kAhead][V];
        if (parts > 0) {
            lse0 = lane < one ? __ldcg(p.part_lse + part_at(lane)) : -INFINITY;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load(k, k < parts, ahead[k]);
        }
        float m = lse0;
        for (int32_t c = 32 + lane; c < parts; c += 32) m = fmaxf(m, __ldcg(p.part_lse + part_at(c)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        float t = 0.f, acc[V];
#pragma unroll
        for (int u = 0; u < V; ++u) acc[u] = 0.f;
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
            for (int32_t c1 = kAhead; c1 < parts; c1 += kAhead) {
                if (c1 % 32 == 0) {
                    const float l = c1 + lane < parts ? __ldcg(p.part_lse + part_at(c1 + lane)) : -INFINITY;
                    w = l == -INFINITY ? 0.f : expf(l - m);
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) load(c1 + k, c1 + k < parts, ahead[k]);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, (c1 + k) & 31);
                    t += wk;
#pragma unroll
                    for (int u = 0; u < V; ++u) acc[u] = fmaf(wk, ahead[k][u], acc[u]);
                }
            }
        }
        const bool empty = !(t > 0.f);
        const float inv = empty ? 0.f : 1.f / t;
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
        if (lane == 0 && st.dv == 0 && p.lse) p.lse[orow] = empty ? -INFINITY : m + logf(t);
    }
}

}  // namespace

cudaError_t launch_tree_join(const TreeAttnParams& p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    // about one wave of warps: a warp then takes several rows of a large call, one of a small one
    const int64_t wave = (int64_t)device_sm_count() * 4, tiles = (int64_t)p.B * p.Hkv * p.n_sub;
    const int64_t most = (p.rows + kWarps - 1) / kWarps;
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv), (unsigned)p.n_sub,
                       (unsigned)std::max<int64_t>(1, std::min(most, (wave + tiles - 1) / tiles)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // a lane's floats: the narrowest that cover the partial's row (DV is a multiple of 16)
    if (p.DV <= 64) return cudaLaunchKernelEx(&cfg, tree_join_kernel<2>, p);
    if (p.DV <= 128) return cudaLaunchKernelEx(&cfg, tree_join_kernel<4>, p);
    if (p.DV <= 256) return cudaLaunchKernelEx(&cfg, tree_join_kernel<8>, p);
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<16>, p);
}

}  // namespace dflash
