// Attention over an e4m3 cache on the tensor cores for few query rows per KV head: single tokens, drafted blocks, small
// trees; and for head_dim above 256. The transposed products of the block attention (tc_attn.cu), whose cost is the rows'
// and not a tile of 128 of them, all in 8 bits:
//
//   S^T [128 keys x N]          = K (Q_hi + Q_lo)^T          e4m3 x e4m3
//   O^T [128 dims x N] (D/128) += V^T (P_1 + P_2 + P_3)^T    e4m3 x e5m2
//
// K and V are operands as they come from the cache, V's stages as MN-major ones, so that a byte of the cache is written to
// shared memory once and read from it once. Bound: the bytes, where requests are long: one token each of 32 requests of 1k
// to 32k keys (32/8 heads of 128, 1.11 GB) takes 183 to 197 us, 5.6 to 6.1 TB/s. At that rate an SM takes in 23
// bytes a cycle and its shared memory moves 128, of which widening V to 16 bits took 6 a byte (262 us, the MMAs waiting for shared
// memory). Blocks of 9 queries of 32/4 heads of 512 over 60k to 131k keys of 4 requests (1.57 GB) take 346 to 353 us, 4.5 TB/s: 72
// rows leave rings of 2 stages each, and the softmax of a tile and its MMAs partly wait for each other.
//
// P' (cache8_tc.cuh) in three e5m2 numbers: as fp16, whose upper byte an e5m2 number is, P' loses its upper byte twice and
// the rest is rounded to a third: 9 significant bits, off by 2^-9 like bf16, all in one scale, as e5m2 has fp16's range.
// The largest P' of a row is kept in [2^11, 2^15] (the maximum moves when a score exceeds it by 2^4), e5m2's
// steps end at 2^-16: 2^-27 of the largest or less, so that many small probabilities beside a large one keep their weight.
//
// N is the rows rounded up to 16, at most 80. Up to 32 rows the parts of Q and of P lie side by side in one operand, K's or
// V's stage is read once, and the softmax or the output adds the results; above, the parts are multiplied one after the other
// into the same columns. The deal of key tiles to CTAs, the masks and the join of split requests are tree attention's
// (tree_attn.cuh, tree_join.cu).
//
// Softmax: a thread is a key of the tile, warps w and w + 4 share keys and take alternate groups of 8 rows; a page's scales
// are its own registers. (Even tiles to warps 0-3 and odd ones to 4-7, with outputs of their own, took 225 us in place of 198
// for the 32 single tokens.) The row maxima are lazy: a tile that moves none costs one comparison a score and one barrier. Row
// sums stay in the threads' registers to the end of the piece. P is MN-major with a 32-byte swizzle: a thread writes 8 rows
// of a part in one 8-byte store.
//
// MMA order: S(0), S(1), then for every tile t: O += P(t) V and S(t + 2), a chunk of 128 dims of each in turn. V rows that
// no query sees are zeroed in the two tiles that can hold some: 0 x NaN would reach every row.
//
// Every mbarrier wait is bounded (p.wait_ns): on expiry the kernel records DFLASH_DEVERR_TIMEOUT, waits (bounded) for
// its own copies and MMAs, frees TMEM and returns.
#include "cache8_tc.cuh"

namespace dflash {
namespace {

using namespace tc8;

// In place of the shift of a row that has seen no key yet: any score of one exceeds the threshold with it, and -inf stays.
constexpr float kUnseen = 3e38f;
constexpr float kRescaleThresh = 4.0f;  // a row's maximum moves when a score exceeds it by more
constexpr float kLift = 11.0f;          // what P' is scaled by, in the exp2 domain
constexpr int kParts = 3;               // of P

template <int N>
struct FewMisc {
    Pipe pipe;
    alignas(16) float c[N];      // of a row: its scale times the softmax's, in the exp2 domain; 0: no query
    alignas(16) float shift[N];  // kLift - its maximum
    alignas(16) float alpha[N];  // what its sum and output are multiplied by
    float m[N];                  // its maximum of x + log2 vs
    float red[4][N];
    float inv[N];
    int32_t node[N];             // its query among the tile's
    // then lo [npt], masks of the request's own keys [npt][(T + 31) / 32]
};

__device__ __forceinline__ void load_row8(const float* src, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// What N = 16 NQ rows make of the operands. Up to 32 rows the parts of Q and of P lie side by side, their rows one behind the
// other, and TMEM's 512 columns hold two S^T and O^T of every part for any head_dim; above, a part is multiplied after
// the other. P lies in atoms of 32 rows x 128 keys, in two buffers (one, which leaves 80 rows of 512 dims 6 stages in place of 4, took
// 362 us in place of 355 for the blocks of 9).
template <int NQ>
struct FewShape {
    static constexpr int N = 16 * NQ;
    static constexpr bool kStack = NQ <= 2;
    static constexpr int kSN = kStack ? 2 * N : N;       // TMEM columns of an S^T
    static constexpr int kON = kStack ? kParts * N : N;  // and of 128 dims of O^T
    static constexpr int kPBytes = kStack ? (kParts * N + 31) / 32 * 4096 : kParts * ((N + 31) / 32) * 4096;
};
static_assert(2 * FewShape<2>::kSN + 4 * FewShape<2>::kON <= 512 && 2 * FewShape<5>::kSN + 4 * FewShape<5>::kON <= 512, "TMEM");

template <int NQ>  // groups of 16 rows
__global__ void __launch_bounds__(kThreads, 1)
    cache8_attn_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ TreeAttnParams p, const Shape x)
{
    using F = FewShape<NQ>;
    constexpr int N = F::N, kSN = F::kSN, kON = F::kON, kPBytes = F::kPBytes;
    constexpr bool kStack = F::kStack;
    constexpr int kOwn = NQ;  // groups of 8 rows per thread, at most
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer, so that the compiler knows what is in shared memory)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const int32_t kc_n = (p.D + 127) / 128;  // chunks of 128 dims
    uint8_t* q_s = smem;
    uint8_t* p_s = smem + (size_t)kc_n * 2 * N * 128;
    uint8_t* k_ring = p_s + 2 * kPBytes;
    uint8_t* v_ring = k_ring + (size_t)x.k_stages * kStageBytes;
    FewMisc<N>& sm = *reinterpret_cast<FewMisc<N>*>(v_ring + (size_t)x.r_stages * kStageBytes);
    Pipe& ms = sm.pipe;
    int32_t* lo_s = reinterpret_cast<int32_t*>(&sm + 1);
    uint32_t* anc_s = reinterpret_cast<uint32_t*>(lo_s + p.npt);
    volatile int* abort_flag = &ms.abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t range = blockIdx.x / p.n_sub, sub = blockIdx.x % p.n_sub;
    const SubTile st = sub_tile(p, sub);
    const int32_t node0 = st.rt * p.npt;

    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, p.err, p.wait_ns));
    };

    if (tid == 0) init_pipe(ms, 1, 1, 8);
    if (warp == kMmaWarp) {
        tmem_alloc(&ms.tmem, 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();  // the kernel before may still run until here
    PieceWalk w;  // the scale warp's
    if (warp == kScaleWarp) {
        w.start(p, range);
        list_pieces(p, w, ms);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cudaTriggerProgrammaticLaunchCompletion();  // the join grid may take its place; it waits for this one to end
    const uint32_t tmem = ms.tmem, tmem_o = tmem + 2 * kSN;
    bool ok = true;

    if (warp < 8) {
        take_registers();
        // ------------------------------------------------------------------ softmax and output
        const int half = warp >> 2, kl = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int words = (p.T + 31) / 32;
        // this key's 32-byte row of every 32-row atom of P, its two 16-byte halves swapped for keys 4-7 of a group
        uint8_t* p_row = p_s + (kl >> 3) * 256 + (kl & 7) * 32;
        const int swz = (kl & 4) << 2;
        uint32_t s_phase = 0, o_phase = 0, q_phase = 0;  // bit b of s_phase, o_phase: parity of next S, product of buffer b
        RingPos sc{0, 0u};
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = wait_all(bar, parity);
            tc_fence_after();
        };
        int32_t masks_of = -1;  // the request whose queries' masks are in shared memory
        // A failed wait ends the computation, not the walk: the barriers below are met by every thread.
        each_piece(p, w, node0, ms, false, [&](const Piece& pc) {
            const int32_t live = min(p.npt, pc.n - node0) * p.Gc;  // rows with a query
            const int32_t steps = pc.tiles;
            const int32_t ctx = pc.ctx;
            const int32_t first_key = pc.first_key, end_key = first_key + steps * kTile;
            const int32_t win_end = p.window > 0 ? ctx + pc.n - p.window : 0;  // keys from here on: no window's edge
            if ((end_key > ctx || first_key < win_end) && masks_of != pc.b) {
                masks_of = pc.b;  // (the KV heads of a request share them)
                // (the barrier that ended the last piece keeps its masks from being overwritten)
                tree_load_parents(p, pc.b, pc.n, ms.par, tid, 256);
                named_bar_sync_256();
                tree_walk_nodes(p, TreeReq{pc.n, pc.ctx, pc.L, pc.lo, 0, 0, false}, node0, min(p.npt, pc.n - node0), ms.par,
                                anc_s, lo_s, tid, 256);
            }
            wait_warp(&ms.q_full, q_phase);
            if (tid < N) {
                // a row without a query gets P = 0
                const bool on = tid < live;
                sm.c[tid] = on ? ms.q_scale[q_phase][tid] * p.scale * kLog2e : 0.f;
                sm.m[tid] = on ? -INFINITY : kUnseen;
                sm.shift[tid] = on ? kUnseen : -kUnseen;
                sm.node[tid] = min(tid / p.Gc, p.npt - 1);
            }
            q_phase ^= 1u;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_free);
            named_bar_sync_256();
            const int groups = (live + 7) / 8;  // of 8 rows; the rest of N has no query
            float l[kOwn][8];
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
#pragma unroll
                for (int u = 0; u < 8; ++u) l[i][u] = 0.f;
#pragma unroll 1
            for (int32_t t = 0; t < steps; ++t) {
                const int buf = t & 1;
                const int32_t key0 = first_key + t * kTile, key = key0 + kl;
                const bool edge = key0 + kTile > ctx || key0 < win_end;
                const uint32_t s_addr = tmem + (uint32_t)buf * kSN + lanes;
                // (that S(t) is done says that the product of tile t - 2 is, which was issued before it: its P's buffer is free)
                const bool s_here = ready(ms.s_full + buf, (s_phase >> buf) & 1u), sc_here = ready(ms.sc_full + sc.idx, sc.phase);
                if (!__all_sync(0xffffffffu, s_here && sc_here)) {
                    wait_warp(ms.sc_full + sc.idx, sc.phase);
                    wait_warp(ms.s_full + buf, (s_phase >> buf) & 1u);
                }
                tc_fence_after();
                s_phase ^= 1u << buf;
                const float ks = ms.k_scale[sc.idx][kl >> 3], v_log = ms.v_log[sc.idx][kl >> 3],
                            v_inv = ms.v_inv[sc.idx][kl >> 3];
                __syncwarp();
                if (lane == 0) mbar_arrive(ms.sc_free + sc.idx);
                sc.advance(1, kScaleRing);
                // which of this thread's rows see the key
                uint64_t seen = ~0ull;
                if (edge) {
                    const int32_t a = key - ctx;
                    seen = 0;
#pragma unroll 1
                    for (int q = 0; q < 8 * kOwn; ++q) {
                        const int row = (half + 2 * (q >> 3)) * 8 + (q & 7);
                        if (row >= live) continue;
                        const int nd = sm.node[row];
                        const bool vis =
                            a < 0 ? key >= lo_s[nd] : (a < pc.n && ((anc_s[nd * words + (a >> 5)] >> (a & 31)) & 1u));
                        seen |= (uint64_t)vis << q;
                    }
                }
                // The scores of group g of this key: S times (the key's scale times the rows' c), plus log2 vs and `shift`
                const uint64_t ks2 = pack2(ks, ks), log2v = pack2(v_log, v_log);
                auto scaled = [&](const uint32_t (&r)[8], const uint32_t (&r2)[8], int g, uint32_t bits, const float* shift,
                                  float (&y)[8]) {
                    float c[8], sh[8];
                    load_row8(sm.c + g * 8, c);
                    if (shift) load_row8(shift + g * 8, sh);
#pragma unroll
                    for (int u = 0; u < 8; u += 2) {
                        uint64_t v = pack2(u2f(r[u]), u2f(r[u + 1]));
                        if (kStack) v = add2(v, pack2(u2f(r2[u]), u2f(r2[u + 1])));
                        v = fma2(v, mul2(pack2(c[u], c[u + 1]), ks2), log2v);  // (S times the key's scale may leave fp32's range)
                        if (shift) v = add2(v, pack2(sh[u], sh[u + 1]));
                        unpack2(v, y[u], y[u + 1]);
                    }
                    if (edge) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) y[u] = (bits >> u) & 1u ? y[u] : -INFINITY;
                    }
                };
                // z = x + log2 vs + the row's shift, what P' is the power of; -inf where a row does not see the key. Where one
                // exceeds the threshold (any that is seen does on a row's first tile) the rows' maxima move, and z is
                // worked out again.
                float z[kOwn][8];
#pragma unroll 1
                for (int again = 0; again < 2; ++again) {
                    bool need = false;
                    if (ok) {
                        uint32_t r[kOwn][8], r2[kOwn][8];
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) {
                            const int g = half + 2 * i;
                            if (g < groups) {
                                tmem_ld8(s_addr + g * 8, r[i]);
                                if (kStack) tmem_ld8(s_addr + N + g * 8, r2[i]);
                            }
                        }
                        tmem_ld_wait();
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) {
                            const int g = half + 2 * i;
                            if (g < groups) {
                                reg_fence8(r[i]);
                                if (kStack) reg_fence8(r2[i]);
                                scaled(r[i], r2[i], g, (uint32_t)(seen >> (8 * i)), sm.shift, z[i]);
#pragma unroll
                                for (int u = 0; u < 8; u += 2) top = fmaxf(fmaxf(z[i][u], z[i][u + 1]), top);
                            }
                        }
                        need = top > kRescaleThresh + kLift;
                    }
                    if (again > 0) break;
                    need = named_bar_or_256(need);
                    if (!need) break;
#pragma unroll 1
                    for (int i = 0; i < kOwn; ++i) {
                        const int g = half + 2 * i;
                        if (ok && g < groups) {
                            uint32_t r[8], r2[8];
                            tmem_ld8(s_addr + g * 8, r);
                            if (kStack) tmem_ld8(s_addr + N + g * 8, r2);
                            tmem_ld_wait();
                            reg_fence8(r);
                            if (kStack) reg_fence8(r2);
                            float y[8];
                            scaled(r, r2, g, (uint32_t)(seen >> (8 * i)), nullptr, y);
                            const float mx = transpose8<false>(y, lane);
                            if (lane < 8) sm.red[warp & 3][g * 8 + lane] = mx;
                        }
                    }
                    named_bar_sync_256();
                    if (tid < live) {
                        const float mo = sm.m[tid];
                        const float mn = fmaxf(fmaxf(mo, fmaxf(sm.red[0][tid], sm.red[1][tid])),
                                               fmaxf(sm.red[2][tid], sm.red[3][tid]));
                        sm.m[tid] = mn;
                        sm.shift[tid] = mn == -INFINITY ? kUnseen : kLift - mn;
                        sm.alpha[tid] = mo == -INFINITY ? 0.f : ex2(mo - mn);
                    }
                    named_bar_sync_256();
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) {
                        const int g = half + 2 * i;
                        if (g < groups) {
                            float a[8];
                            load_row8(sm.alpha + g * 8, a);
#pragma unroll
                            for (int u = 0; u < 8; ++u) l[i][u] *= a[u];
                        }
                    }
                    // O holds the tiles before this one once their product is done: only a rescale waits for it here
                    if (t > 0) {
                        wait_warp(ms.p_free + (buf ^ 1), (o_phase >> (buf ^ 1)) & 1u);
                        if (ok) {
#pragma unroll 1
                            for (int cg = half; cg < kc_n * groups; cg += 2) {
                                const int c = cg / groups, g = cg - c * groups;
                                float a[8];
                                load_row8(sm.alpha + g * 8, a);
#pragma unroll
                                for (int i = 0; i < kON / N; ++i) {
                                    const uint32_t at = tmem_o + c * kON + i * N + g * 8 + lanes;
                                    uint32_t o[8];
                                    tmem_ld8(at, o);
                                    tmem_ld_wait();
                                    reg_fence8(o);
#pragma unroll
                                    for (int u = 0; u < 8; ++u) o[u] = f2u(u2f(o[u]) * a[u]);
                                    tmem_st8(at, o);
                                }
                            }
                            tmem_st_wait();
                        }
                    }
                }
                if (t > 0) o_phase ^= 1u << (buf ^ 1);  // (the phase of the tile before; never two behind)
                if (ok) {
                    const uint64_t inv2 = pack2(v_inv, v_inv);
                    uint8_t* p_buf = p_row + buf * kPBytes;
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) {
                        const int g = half + 2 * i;
                        if (g < groups) {
                            __half2 h[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const float a = ex2(z[i][2 * u]), b = ex2(z[i][2 * u + 1]);
                                unpack2(fma2(pack2(a, b), inv2, pack2(l[i][2 * u], l[i][2 * u + 1])), l[i][2 * u],
                                        l[i][2 * u + 1]);
                                h[u] = __floats2half2_rn(a, b);
                            }
#pragma unroll
                            for (int part = 0; part < kParts; ++part) {
                                uint32_t w32[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    w32[u] = *reinterpret_cast<const uint32_t*>(&h[u]);
                                    if (part == kParts - 1) {
                                        w32[u] += 0x00800080u;  // to nearest (P is not negative)
                                    } else {
                                        const uint32_t top = w32[u] & 0xFF00FF00u;
                                        h[u] = __hsub2(h[u], *reinterpret_cast<const __half2*>(&top));
                                    }
                                }
                                const int at = (kStack ? part * N : 0) + g * 8;  // row of the operand
                                *reinterpret_cast<uint2*>(p_buf + (kStack ? 0 : part * (kPBytes / kParts)) + (at >> 5) * 4096 +
                                                          ((at & 16) ^ swz) + (at & 15)) =
                                    make_uint2(__byte_perm(w32[0], w32[1], 0x7531), __byte_perm(w32[2], w32[3], 0x7531));
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ms.p_full + buf);
            }
            wait_warp(ms.p_free + ((steps - 1) & 1), (o_phase >> ((steps - 1) & 1)) & 1u);
            o_phase ^= 1u << ((steps - 1) & 1);
            // ---------------------------------------------------------------- output
            const bool whole = pc.whole != 0;
            const int64_t prow = tree_part_row(p, range, sub, pc.slot);
            const int64_t orow = ((int64_t)pc.b * p.T + node0) * p.Hq + pc.g * p.G + st.gc * p.Gc;  // of row 0
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const int g = half + 2 * i;
                if (g < groups) {
                    const float sum = transpose8<true>(l[i], lane);
                    if (lane < 8) sm.red[warp & 3][g * 8 + lane] = sum;
                }
            }
            tc_fence_before();
            named_bar_sync_256();
            tc_fence_after();
            if (tid < live) {
                const float tot = (sm.red[0][tid] + sm.red[1][tid]) + (sm.red[2][tid] + sm.red[3][tid]);
                const float lse = tree_row_lse((sm.m[tid] - kLift + log2f(tot)) * kLn2, tot, whole);
                sm.inv[tid] = tree_inv_sum(tot, whole) * ms.v_ref;
                if (!whole)
                    p.part_lse[prow + tid] = lse;
                else if (p.lse)
                    p.lse[orow + (int64_t)sm.node[tid] * (p.Hq - p.Gc) + tid] = lse;
            }
            named_bar_sync_256();
            if (ok) {
#pragma unroll 1
                for (int cg = half; cg < kc_n * groups; cg += 2) {
                    const int c = cg / groups, g = cg - c * groups;
                    const int32_t d = c * 128 + (warp & 3) * 32 + lane;
                    uint32_t o[kON / N][8];
#pragma unroll
                    for (int k = 0; k < kON / N; ++k) tmem_ld8(tmem_o + c * kON + k * N + g * 8 + lanes, o[k]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < kON / N; ++k) reg_fence8(o[k]);
                    if (d < p.D) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int row = g * 8 + u;
                            if (row < live) {
                                float v = u2f(o[0][u]);
#pragma unroll
                                for (int k = 1; k < kON / N; ++k) v += u2f(o[k][u]);
                                v *= sm.inv[row];
                                if (!whole)
                                    p.part_out[(prow + row) * p.DV + d] = v;
                                else
                                    static_cast<__nv_bfloat16*>(
                                        p.out)[(orow + (int64_t)sm.node[row] * (p.Hq - p.Gc) + row) * p.D + d] =
                                        __float2bfloat16_rn(v);
                            }
                        }
                    }
                    __syncwarp();  // the next load takes the whole warp
                }
            }
            tc_fence_before();
            named_bar_sync_256();  // O, the sums and the masks are read before the next piece's steps
        });
        tc_fence_before();
        asm volatile("barrier.sync 0;" ::: "memory");  // every role is done (the end of the others' branch)
        if (ms.far != 0) far_pieces(p, x.page_magic, range, sub, ms.v_ref, ms.par, lo_s, anc_s);
    } else {
        give_registers();
        if (warp == kKWarp) {
            produce(p, x, w, node0, ms, &tm_k, k_ring, ms.k_full, ms.k_empty, x.k_stages, wait_all);
        } else if (warp == kVWarp) {
            produce(p, x, w, node0, ms, &tm_v, v_ring, ms.r_full, ms.r_empty, x.r_stages, wait_all);
        } else if (warp == kScaleWarp) {
            fetch_scales(p, x, w, node0, ms, wait_all);
        } else if (warp >= kConvertWarp) {
            split_all(p, x, w, st, node0, ms, q_s, wait_all);
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------------ MMA issuer
            // Everything about an MMA but the issue itself is the same for the whole warp, so that it lies in uniform
            // registers, where the instruction wants it.
            constexpr uint32_t idesc_s = idesc_f8(128, kSN, 0, 0, 0);
            constexpr uint32_t idesc_o = idesc_f8(128, kON, 1, 1, 1);
            const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024), k_desc = sw128_desc(smem_u32(k_ring), 16, 1024),
                           v_desc = sw128_desc(smem_u32(v_ring), 8192, 1024), p_desc = sw32_desc(smem_u32(p_s), 4096, 256);
            constexpr uint32_t q_chunk = N * 8;  // hi, then lo of a chunk, in 16-byte units
            RingPos kp{0, 0u}, vp{0, 0u};
            uint32_t q_phase = 0, p_phase = 0;  // p_phase: bit b = parity of the next P in buffer b
            each_piece(p, w, node0, ms, false, [&](const Piece& pc) {
                if (!ok) return;
                const int32_t steps = pc.tiles;
                ok = wait_all(&ms.q_full, q_phase);
                if (!ok) return;
                q_phase ^= 1u;
                // chunk c of S(t)
                auto scores = [&](int32_t t, int32_t c) {
                    ok = wait_all(ms.k_full + kp.idx, kp.phase);
                    if (!ok) return;
                    const uint32_t d = tmem + (uint32_t)(t & 1) * kSN;
                    const uint64_t kd = k_desc + (uint32_t)kp.idx * (kStageBytes / 16), qd = q_desc + c * 2 * q_chunk;
                    const int32_t part = (min(128, p.D - c * 128) + 31) / 32;  // steps of 32 dims; the rest is zeros
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk < part) {
                                tc_mma_f8(d, kd + 2 * kk, qd + 2 * kk, idesc_s, (c > 0 || kk > 0) ? 1u : 0u);
                                if (!kStack) tc_mma_f8(d, kd + 2 * kk, qd + q_chunk + 2 * kk, idesc_s, 1u);
                            }
                        }
                        tc_commit(ms.k_empty + kp.idx);
                        if (c == kc_n - 1) tc_commit(ms.s_full + (t & 1));
                        if (c == kc_n - 1 && t == steps - 1) tc_commit(&ms.q_free);
                    }
                    __syncwarp();
                    kp.advance(1, x.k_stages);
                };
                // chunk c of O += P(t) V
                auto values = [&](int32_t t, int32_t c) {
                    const uint64_t pd = p_desc + (uint32_t)(t & 1) * (kPBytes / 16);
                    const int32_t key0 = pc.first_key + t * kTile;
                    ok = wait_all(ms.r_full + vp.idx, vp.phase);
                    if (!ok) return;
                    if (key0 < pc.lo || key0 + kTile > pc.L) {
                        uint8_t* stage = v_ring + (size_t)vp.idx * kStageBytes;
                        const int32_t from = pc.lo - key0, to = pc.L - key0;  // the visible rows
                        for (int32_t i = lane; i < kTile * 8; i += 32)
                            if ((i >> 3) < from || (i >> 3) >= to)
                                *reinterpret_cast<uint4*>(stage + i * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const uint64_t vd = v_desc + (uint32_t)vp.idx * (kStageBytes / 16);
                    if (elect_one()) {
#pragma unroll
                        for (int part = 0; part < (kStack ? 1 : kParts); ++part)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma_f8(tmem_o + c * kON, vd + kk * 256, pd + part * (kPBytes / kParts / 16) + kk * 64,
                                          idesc_o, (t > 0 || part > 0 || kk > 0) ? 1u : 0u);
                        tc_commit(ms.r_empty + vp.idx);
                        if (c == kc_n - 1) tc_commit(ms.p_free + (t & 1));
                    }
                    __syncwarp();
                    vp.advance(1, x.r_stages);
                };
#pragma unroll 1
                for (int32_t t = 0; t < min(2, steps) && ok; ++t)
#pragma unroll 1
                    for (int32_t c = 0; c < kc_n && ok; ++c) scores(t, c);
                // The chunks of O += P(t) V and of S(t + 2) in turn: the stages of both rings go evenly, where a tile of many
                // dims would take all of one at once and wait for the copies behind them.
#pragma unroll 1
                for (int32_t t = 0; t < steps && ok; ++t) {
                    ok = wait_all(ms.p_full + (t & 1), (p_phase >> (t & 1)) & 1u);
                    if (!ok) break;
                    p_phase ^= 1u << (t & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int32_t c = 0; c < kc_n && ok; ++c) {
                        values(t, c);
                        if (ok && t + 2 < steps) scores(t + 2, c);
                    }
                }
            });
            // our MMAs end before TMEM is freed
            if (elect_one()) {
                tc_commit(&ms.drain);
                const unsigned long long t0 = globaltimer();
                while (!mbar_test_wait(&ms.drain, 0) && globaltimer() - t0 < kDrainNs) {
                }
            }
            __syncwarp();
        }
        // ---------------------------------------------------------------------- teardown
        tc_fence_before();
        asm volatile("barrier.sync 0;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int NQ>
cudaError_t launch_nq(const CUtensorMap& tk, const CUtensorMap& tv, const TreeAttnParams& p, Shape x, cudaStream_t stream)
{
    using F = FewShape<NQ>;
    const int32_t fixed = (p.D + 127) / 128 * 2 * F::N * 128 + 2 * F::kPBytes + 1024;
    const int32_t misc = (int32_t)sizeof(FewMisc<F::N>) + p.npt * 4 * (1 + (p.T + 31) / 32);
    const int32_t stages = (kSmemMax - fixed - misc) / kStageBytes;
    if (stages < 2) return cudaErrorInvalidConfiguration;
    x.k_stages = std::min(kMaxStages, (stages + 1) / 2);
    x.r_stages = std::min(kMaxStages, stages / 2);
    auto* kernel = cache8_attn_few_kernel<NQ>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.ranges * p.n_sub));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = fixed + (x.k_stages + x.r_stages) * kStageBytes + misc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];  // set-up beside the end of the kernel before
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, tk, tv, p, x);
}

}  // namespace

cudaError_t tc8::launch_few(const CUtensorMap& tk, const CUtensorMap& tv, const TreeAttnParams& p, Shape x,
                            cudaStream_t stream)
{
    switch ((p.rows + 15) / 16) {
    case 1: return launch_nq<1>(tk, tv, p, x, stream);
    case 2: return launch_nq<2>(tk, tv, p, x, stream);
    case 3: return launch_nq<3>(tk, tv, p, x, stream);
    case 4: return launch_nq<4>(tk, tv, p, x, stream);
    default: return launch_nq<5>(tk, tv, p, x, stream);
    }
}

}  // namespace dflash
