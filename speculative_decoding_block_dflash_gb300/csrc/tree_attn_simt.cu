// Tree attention on the CUDA cores: the fp32 path, and bf16 for layouts that the tensor-core kernel does not
// take.
//
//   s_ij = scale <q_i, k_j> over the keys that node i sees, out_i = sum_j softmax(s_i)_j v_j
//
// A CTA of 256 threads owns a tile of up to 64 query rows (node x head) and streams its range's key tiles of 64
// keys once. Products are register-tiled: a thread holds R rows x 4 keys of the scores and R rows x 4 dims of
// every 64-dim chunk of the output, so each value read from shared memory feeds R to 4 R FMAs; R is 4, or 2 or
// 1 where a KV head has no more than 32 or 16 rows, and warps whose rows hold no node only load (one node's 4
// rows a KV head, 4 requests of 8192 keys, D = 128: 335 us in tiles of 64, 207 of 16, 111 with the idle warps
// out of shared memory's way). K and V pass through two shared buffers of 64 keys x 64 dims (widened to fp32);
// the next chunk's global loads are in flight in registers while the current one is used, and one barrier per
// chunk is enough. The softmax is online: running maximum and sum per row in fp32, replicated over the row's 16
// threads. Bound: shared memory's bandwidth for full tiles (24 wavefronts per 64 FMAs of a warp), the loads in
// flight for few rows. Measured, fp32, 4 requests of 8192 keys, 32/8 heads of 128: 64 nodes 1270 us (24
// TFLOP/s), 16 nodes 335 (23), 1 node 111 (2.4 TB/s); 2 requests of 4096 keys, 16 nodes, 32/4 heads of 512 312
// (26 TFLOP/s), 32/16 heads of 256 236 (17). (Tiles of 128 rows reach 29 TFLOP/s at D = 128, but one request of
// 300 keys takes 55 us in place of 41.)
#include <cmath>

#include "tree_attn.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;
constexpr int kLd = 68;  // floats per shared row of 64: 16-byte loads of 8 rows fall on distinct banks

struct SimtTreeSmem {
    static int q_ld(int D) { return (D + 63) / 64 * 64 + 4; }
    static size_t bytes(int D, int rows)
    {
        return sizeof(float) * ((size_t)rows * (q_ld(D) + kLd) + 2 * kKeys * kLd) +
               sizeof(int32_t) * (DFLASH_MAX_TREE_NODES + rows + rows * (DFLASH_MAX_TREE_NODES / 32));
    }
};

// 16 values of a 64 x 64 chunk for this thread: row tid / 4, dims 16 (tid % 4) .. +15 (as four float4)
__device__ __forceinline__ void fetch16(const TreeAttnParams& p, const void* base, int64_t off, bool live, int d0,
                                        float (&v)[16])
{
#pragma unroll
    for (int u = 0; u < 16; ++u) v[u] = 0.f;
    if (!live || d0 >= p.D) return;  // D is a multiple of 16
    if (p.dtype == DFLASH_BF16) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off + d0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 w = __ldg(s + h);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[h * 8 + 2 * u] = __uint_as_float(x[u] << 16);
                v[h * 8 + 2 * u + 1] = __uint_as_float(x[u] & 0xFFFF0000u);
            }
        }
    } else {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off + d0);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float4 w = __ldg(s + h);
            v[4 * h] = w.x;
            v[4 * h + 1] = w.y;
            v[4 * h + 2] = w.z;
            v[4 * h + 3] = w.w;
        }
    }
}

template <int NC, int R>  // 64-dim chunks, rows per thread
__global__ void __launch_bounds__(kThreads, simt_ctas_per_sm(NC * 64, 16 * R))
    tree_attn_simt_kernel(const TreeAttnParams p)
{
    constexpr int kRows = 16 * R;
    extern __shared__ float smem[];
    const int q_ld = NC * 64 + 4;
    float* Qs = smem;                      // [kRows][q_ld]
    float* Cs = Qs + kRows * q_ld;         // [2][kKeys][kLd] K or V chunk
    float* Ps = Cs + 2 * kKeys * kLd;      // [kRows][kLd]
    int32_t* par_s = reinterpret_cast<int32_t*>(Ps + kRows * kLd);
    int32_t* lo_s = par_s + DFLASH_MAX_TREE_NODES;
    uint32_t* anc_s = reinterpret_cast<uint32_t*>(lo_s + kRows);

    const int tid = threadIdx.x;
    const int ty = tid >> 4, tx = tid & 15;
    const int32_t range = blockIdx.x / p.n_sub, sub = blockIdx.x % p.n_sub;
    const SubTile st = sub_tile(p, sub);
    const int32_t node0 = st.rt * p.npt;
    const int words = (p.T + 31) / 32;
    const int lr = tid >> 2, ld0 = (tid & 3) * 16;  // this thread's part of a chunk load

    cudaTriggerProgrammaticLaunchCompletion();  // the join grid may start; it waits for this one to end
    PieceWalk w;
    for (w.start(p, range); !w.done(); w.next(p)) {
        const int32_t b = w.b, g = w.g, n = w.req.n, ctx = w.req.ctx, L = w.req.L;
        if (node0 >= n) continue;
        const int32_t live = min(p.npt, n - node0) * p.Gc;  // rows with a node
        __syncthreads();                                    // the last piece is done with shared memory
        tree_load_parents(p, b, n, par_s, tid, kThreads);
        for (int c = 0; c < NC; ++c) {
            const int d = c * 64 + ld0;
            float v[16];
            const int32_t node = node0 + lr / p.Gc, head = g * p.G + st.gc * p.Gc + lr % p.Gc;
            fetch16(p, p.q, (((int64_t)b * p.T + node) * p.Hq + head) * p.D, lr < live, d, v);
            if (lr >= kRows) continue;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                *reinterpret_cast<float4*>(Qs + lr * q_ld + d + 4 * u) =
                    make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        }
        __syncthreads();
        tree_walk_nodes(p, w.req, node0, min(p.npt, n - node0), par_s, anc_s, lo_s, tid, kThreads);
        // (the first chunk's barrier below makes the walk's results visible before the first mask)

        const bool idle = (tid >> 5) * 2 * R >= live;  // this warp's rows have no node: it only loads
        float o[NC][R][4], m[R], l[R];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[c][i][u] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
        // global offset of this thread's load row in tile t, or -1 for keys that nobody sees or a bad page
        auto key_off = [&](int32_t t) -> int64_t {
            const int32_t j = (w.req.tile0 + t) * kKeys + lr;
            if (t >= w.t1 || j < w.req.lo || j >= L) return -1;
            const int32_t page = __ldg(p.page_table + (int64_t)b * p.max_pages + j / p.page_size);
            if (page < 0 || page >= p.num_pages) {
                raise_error(p.err, DFLASH_DEVERR_PAGE_ID);
                return -1;
            }
            return (int64_t)page * p.sp + (int64_t)(j % p.page_size) * p.ss + (int64_t)g * p.sh;
        };
        int buf = 0;
        float nxt[16];
        int64_t off = key_off(w.t0);
        fetch16(p, p.k, off, off >= 0, ld0, nxt);
        auto publish = [&]() -> const float* {
            float* dst = Cs + buf * kKeys * kLd;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                *reinterpret_cast<float4*>(dst + lr * kLd + ld0 + 4 * u) =
                    make_float4(nxt[4 * u], nxt[4 * u + 1], nxt[4 * u + 2], nxt[4 * u + 3]);
            buf ^= 1;
            __syncthreads();
            return dst;
        };
        for (int32_t t = w.t0; t < w.t1; ++t) {
            const int32_t k0 = (w.req.tile0 + t) * kKeys;
            float s[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                const float* ks = publish();
                if (c + 1 < NC)
                    fetch16(p, p.k, off, off >= 0, (c + 1) * 64 + ld0, nxt);
                else
                    fetch16(p, p.v, off, off >= 0, ld0, nxt);
                if (idle) continue;
#pragma unroll 4
                for (int d = 0; d < 64; d += 4) {
                    float4 qv[R], kv[4];
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        qv[i] = *reinterpret_cast<const float4*>(Qs + (ty * R + i) * q_ld + c * 64 + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * kLd + d);
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                            s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                            s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                            s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
                        }
                }
            }
            const bool edge = k0 + kKeys > ctx || (p.window > 0 && k0 < ctx + n - p.window + 1);
            float alpha[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = ty * R + i;
                if (idle) continue;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    bool vis = true;
                    if (edge) {
                        const int32_t key = k0 + tx + 16 * j;
                        const int nd = row / p.Gc;
                        vis = row < live;
                        if (vis) {
                            const int32_t a = key - ctx;
                            vis = a < 0 ? key >= lo_s[nd]
                                        : (key < L && ((anc_s[nd * words + (a >> 5)] >> (a & 31)) & 1u));
                        }
                    }
                    s[i][j] = vis ? s[i][j] * p.scale : -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[i], mx);
                alpha[i] = m[i] == -INFINITY ? 0.f : expf(m[i] - mn);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = s[i][j] == -INFINITY ? 0.f : expf(s[i][j] - mn);
                    Ps[row * kLd + tx + 16 * j] = e;
                    sum += e;
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[i] = l[i] * alpha[i] + sum;
            }
            const int64_t next_off = key_off(t + 1);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float* vs = publish();
                if (c + 1 < NC)
                    fetch16(p, p.v, off, off >= 0, (c + 1) * 64 + ld0, nxt);
                else
                    fetch16(p, p.k, next_off, next_off >= 0, ld0, nxt);
                if (idle) continue;
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int u = 0; u < 4; ++u) o[c][i][u] *= alpha[i];
#pragma unroll 2
                for (int k = 0; k < kKeys; k += 4) {
                    float4 pv[R], vv[4];
#pragma unroll
                    for (int i = 0; i < R; ++i) pv[i] = *reinterpret_cast<const float4*>(Ps + (ty * R + i) * kLd + k);
#pragma unroll
                    for (int j = 0; j < 4; ++j) vv[j] = *reinterpret_cast<const float4*>(vs + (k + j) * kLd + tx * 4);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float pr[4] = {pv[i].x, pv[i].y, pv[i].z, pv[i].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            o[c][i][0] = fmaf(pr[j], vv[j].x, o[c][i][0]);
                            o[c][i][1] = fmaf(pr[j], vv[j].y, o[c][i][1]);
                            o[c][i][2] = fmaf(pr[j], vv[j].z, o[c][i][2]);
                            o[c][i][3] = fmaf(pr[j], vv[j].w, o[c][i][3]);
                        }
                    }
                }
            }
            off = next_off;
        }
        const bool whole = w.whole();
        const int64_t prow = tree_part_row(p, range, sub, w.slot());
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = ty * R + i;
            if (row >= live) continue;
            const float inv = tree_inv_sum(l[i], whole);
            const float lse = tree_row_lse(m[i] + logf(l[i]), l[i], whole);
            const int32_t node = node0 + row / p.Gc, head = g * p.G + st.gc * p.Gc + row % p.Gc;
            const int64_t orow = ((int64_t)b * p.T + node) * p.Hq + head;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = c * 64 + tx * 4;
                if (d >= p.D) continue;
                const float4 r = make_float4(o[c][i][0] * inv, o[c][i][1] * inv, o[c][i][2] * inv, o[c][i][3] * inv);
                if (!whole) {
                    *reinterpret_cast<float4*>(p.part_out + (prow + row) * p.DV + d) = r;
                } else if (p.dtype == DFLASH_FP32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow * p.D + d) = r;
                } else {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(r.x, r.y), c2 = __floats2bfloat162_rn(r.z, r.w);
                    uint2 pk;
                    pk.x = *reinterpret_cast<const uint32_t*>(&a);
                    pk.y = *reinterpret_cast<const uint32_t*>(&c2);
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * p.D + d) = pk;
                }
            }
            if (tx == 0) {
                if (!whole)
                    p.part_lse[prow + row] = lse;
                else if (p.lse)
                    p.lse[orow] = lse;
            }
        }
    }
}

template <int NC, int R>
cudaError_t launch_nr(const TreeAttnParams& p, cudaStream_t stream)
{
    const size_t smem = SimtTreeSmem::bytes(NC * 64, 16 * R);
    cudaError_t e =
        cudaFuncSetAttribute(tree_attn_simt_kernel<NC, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // (as a programmatic dependent itself, back to back with the last call's join, calls of 22.6 us took 24.5)
    tree_attn_simt_kernel<NC, R><<<p.ranges * p.n_sub, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int NC>
cudaError_t launch_nc(const TreeAttnParams& p, cudaStream_t stream)
{
    return p.rows <= 16 ? launch_nr<NC, 1>(p, stream)
                        : p.rows <= 32 ? launch_nr<NC, 2>(p, stream) : launch_nr<NC, 4>(p, stream);
}

}  // namespace

cudaError_t launch_tree_attn_simt(const TreeAttnParams& p, cudaStream_t stream)
{
    switch (simt_chunks(p.D)) {
    case 1: return launch_nc<1>(p, stream);
    case 2: return launch_nc<2>(p, stream);
    case 4: return launch_nc<4>(p, stream);
    default: return launch_nc<8>(p, stream);
    }
}

}  // namespace dflash
