// Join of the tree attention's partials: a (request, KV head) pair whose key tiles lie in several
// ranges has one normalised partial (o_c, lse_c) per range and row, and
//   m = max_c lse_c, w_c = exp(lse_c - m), out = sum_c w_c o_c / sum_c w_c, lse = m + log(sum_c w_c).
// Pairs that one range holds whole are final already. A request with a bad length or tree size gets its
// zeros here.
//
// A CTA takes kRows rows of one (pair, query tile); a thread owns a float4 of a row, reads the row's chunk lse
// values itself and keeps eight partial loads in flight. Launched as a programmatic
// dependent of the attention kernel.
#include <cmath>

#include "tree_attn.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) tree_join_kernel(const TreeAttnParams p, int32_t rows_per_cta)
{
    __shared__ int64_t sh_first, sh_total;
    cudaGridDependencySynchronize();
    const int32_t pair = blockIdx.x;
    const int32_t b = pair / p.Hkv, g = pair % p.Hkv;
    const int32_t sub = blockIdx.y;
    const SubTile st = sub_tile(p, sub);
    const TreeReq rq = tree_request(p, b);
    const int32_t node0 = st.rt * p.npt;
    if (rq.bad && g == 0 && sub == 0 && blockIdx.z == 0 && threadIdx.x == 0) raise_error(p.err, tree_request_error(p, rq));
    if (rq.nt == 0 && !rq.bad) return;
    if (!rq.bad && node0 >= rq.n) return;
    const int lanes = p.DV / 4;
    const int d_here = min(p.DV, p.D - st.dv * p.DV);
    int32_t r0 = 0, parts = 0;
    if (!rq.bad) {
        if (threadIdx.x < 32) {
            const int64_t before = tree_tiles_before(p, b), all = tree_tiles_before(p, p.B);
            if (threadIdx.x == 0) {
                sh_first = before + (int64_t)g * rq.nt;
                sh_total = all;
            }
        }
        __syncthreads();
        const int64_t total = sh_total;
        const int32_t used = ranges_used(p, total);
        r0 = range_of(total, used, sh_first);
        parts = range_of(total, used, sh_first + rq.nt - 1) - r0 + 1;
        if (parts == 1) return;
    }
    const int32_t n_here = rq.bad ? p.T : rq.n;
    const int32_t live = min(p.npt, n_here - node0) * p.Gc;
    const int32_t row_end = min(live, (int32_t)(blockIdx.z + 1) * rows_per_cta);
    for (int32_t item = blockIdx.z * rows_per_cta * lanes + threadIdx.x; item < row_end * lanes; item += kThreads) {
        const int32_t row = item / lanes, d0 = (item - row * lanes) * 4;
        float m = -INFINITY;
        for (int c = 0; c < parts; ++c)
            m = fmaxf(m, __ldg(p.part_lse + tree_part_row(p, r0 + c, sub, c == 0 ? 1 : 0) + row));
        float t = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m != -INFINITY && d0 < d_here) {
            for (int c0 = 0; c0 < parts; c0 += 8) {
                float w[8];
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int c = c0 + k;
                    const int64_t at = tree_part_row(p, r0 + min(c, parts - 1), sub, c == 0 ? 1 : 0) + row;
                    const float l = c < parts ? __ldg(p.part_lse + at) : -INFINITY;
                    w[k] = l == -INFINITY ? 0.f : expf(l - m);
                    v[k] = w[k] > 0.f ? __ldg(reinterpret_cast<const float4*>(p.part_out + at * p.DV + d0))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    t += w[k];
                    acc.x = fmaf(w[k], v[k].x, acc.x);
                    acc.y = fmaf(w[k], v[k].y, acc.y);
                    acc.z = fmaf(w[k], v[k].z, acc.z);
                    acc.w = fmaf(w[k], v[k].w, acc.w);
                }
            }
        }
        if (d0 >= d_here) continue;
        const bool empty = !(t > 0.f);
        const float inv = empty ? 0.f : 1.f / t;
        const int32_t node = node0 + row / p.Gc, head = g * p.G + st.gc * p.Gc + row % p.Gc;
        const int64_t orow = ((int64_t)b * p.T + node) * p.Hq + head;
        const int64_t o = orow * p.D + st.dv * p.DV + d0;
        if (p.dtype == DFLASH_BF16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            uint2 pk;
            pk.x = *reinterpret_cast<const uint32_t*>(&lo);
            pk.y = *reinterpret_cast<const uint32_t*>(&hi);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) = pk;
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        }
        if (d0 == 0 && st.dv == 0 && p.lse) p.lse[orow] = empty ? -INFINITY : m + logf(t);
    }
}

}  // namespace

cudaError_t launch_tree_join(const TreeAttnParams& p, cudaStream_t stream)
{
    const int32_t rows_per_cta = 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv), (unsigned)p.n_sub, (unsigned)((p.rows + rows_per_cta - 1) / rows_per_cta));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel, p, rows_per_cta);
}

}  // namespace dflash
