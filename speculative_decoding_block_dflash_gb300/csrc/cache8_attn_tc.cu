// Attention over an e4m3 cache on the tensor cores (bf16 queries, head_dim up to 256), for many query rows per KV head:
// prompt chunks and wide trees.
//
//   S [128 rows x 128 keys] = Q_hi K^T + Q_lo K^T    kind::f8f6f4, K's bytes as they come from the cache
//   O [128 rows x DV]      += P [128 x 128] . V      kind::f16, P in TMEM, V widened to fp16 on the way
//
// A query row is a (query, head of the KV head's group), a TMEM lane; the deal of key tiles to CTAs, the masks and the
// join of split requests are tree attention's (tree_attn.cuh, tree_join.cu), the stages of K, Q and V are cache8_tc.cuh's.
//
// TMEM: S0, S1 (128 columns each; P takes the place of its S) and up to 256 of O. MMA order: S(0), S(1), then for every tile
// t: O += P(t) V, S(t + 2). Two softmax threads share a row's tile, 64 keys each, and exchange one maximum.
//
// Bound: the chain of one tile. 128 rows x 128 keys x 128 dims take some 2400 cycles, the MMAs 1072 of them and the exponentials
// 1024; the widening of V takes about as long beside them. Trees of 32 nodes on 8 requests of 2k to 16k keys (32/8
// heads of 128) take 70 us, 34 GFLOP and 154 MB at 490 TFLOP/s and 2.2 TB/s, chunks of 256 queries of 2 requests of 8k to
// 16k keys 149 us, 101 GFLOP at 673 TFLOP/s.
//
// Every mbarrier wait is bounded (p.wait_ns): on expiry the kernel records DFLASH_DEVERR_TIMEOUT, waits (bounded) for
// its own copies and MMAs, frees TMEM and returns.
#include <algorithm>
#include <mutex>

#include "cache8_tc.cuh"

namespace dflash {
namespace {

using namespace tc8;

constexpr int kSoftmax = 256;  // warps 0-7
constexpr int kOCol = 256;     // first TMEM column of O
constexpr float kRescaleThresh = 8.0f;  // a row's maximum moves when a score exceeds it by more
constexpr float kLift = 7.0f;           // P' <= 2^(8 + 7) < 65504; fp16's steps of 2^-24 are 2^-31 of the largest, or less

struct TcMisc {
    Pipe pipe;
    float mx[2][2][128];  // row maxima of tile t over half of its keys, in [t % 2]
    float l[2][128];
    // then lo [npt], masks of the request's own keys [npt][(T + 31) / 32]
};

template <int DV>
__global__ void __launch_bounds__(kThreads, 1)
    cache8_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ TreeAttnParams p, const Shape x)
{
    constexpr int kVN = DV == 64 ? 64 : 128;     // dims of a V stage
    constexpr int kVKeys = DV == 64 ? 128 : 64;  // and its keys
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer, so that the compiler knows what is in shared memory)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const int32_t kc_n = (p.D + 127) / 128;  // K stages per tile, of 128 dims
    const uint32_t q_chunk_bytes = (uint32_t)x.q_rows * 128;
    uint8_t* q_s = smem;
    uint8_t* k_ring = smem + 2 * (size_t)kc_n * q_chunk_bytes;
    uint8_t* r_ring = k_ring + (size_t)x.k_stages * kStageBytes;
    uint8_t* v_ring = r_ring + (size_t)x.r_stages * kStageBytes;
    TcMisc& sm = *reinterpret_cast<TcMisc*>(v_ring + (size_t)x.v_stages * kStageBytes);
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

    auto wait_one = [&](uint64_t* bar, uint32_t parity) -> bool {
        return wait_bar(bar, parity, abort_flag, p.err, p.wait_ns);
    };

    if (tid == 0) init_pipe(ms, kConverters, 8, 4);
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
    const uint32_t tmem = ms.tmem;
    bool ok = true;

    if (warp < 8) {
        take_registers();
        // ------------------------------------------------------------------ softmax and output
        // Warps w and w + 4 share TMEM lanes, that is rows: a row's tile is split between two threads, of its first and
        // its last 64 keys.
        const int half = warp >> 2;
        const int row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int words = (p.T + 31) / 32;
        uint32_t s_phase = 0, o_phase = 0, q_phase = 0;  // bit b of s_phase, o_phase: parity of the next S, product of buffer b
        RingPos sc{0, 0u};
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = wait_all(bar, parity);
            tc_fence_after();
        };
        // a softmax warp's part of P is in TMEM
        auto arrive = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
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
                tree_load_parents(p, pc.b, pc.n, ms.par, tid, kSoftmax);
                named_bar_sync_256();
                tree_walk_nodes(p, TreeReq{pc.n, pc.ctx, pc.L, pc.lo, 0, 0, false}, node0, min(p.npt, pc.n - node0), ms.par, anc_s, lo_s, tid, kSoftmax);
                named_bar_sync_256();
            }
            const bool live_row = row < live;
            const bool busy = (warp & 3) * 32 < live;  // this warp has a row with a query
            const int32_t nd = row / p.Gc;
            const uint32_t* anc = anc_s + nd * words;
            const uint32_t o_addr = tmem + kOCol + lanes;
            const int32_t d_here = min(DV, p.D);
            const int32_t d0 = half * (DV / 2), d1 = min(d_here, d0 + DV / 2);  // this thread's share of O's columns
            float m2 = -INFINITY, l = 0.f;  // the row's maximum of x + log2 vs, and 2^kLift times the sum over this thread's keys
            wait_warp(&ms.q_full, q_phase);
            const float c = live_row ? ms.q_scale[q_phase][row] * p.scale * kLog2e : 1.f;
            const float not_a_row = c - c;  // 0, or NaN
            q_phase ^= 1u;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_free);
#pragma unroll 1
            for (int32_t t = 0; t < steps; ++t) {
                const int buf = t & 1;
                const int32_t key0 = first_key + t * kTile;
                const bool edge = key0 + kTile > ctx || key0 < win_end;
                const uint32_t s_addr = tmem + (uint32_t)buf * 128 + lanes;
                const bool s_here = ready(ms.s_full + buf, (s_phase >> buf) & 1u), sc_here = ready(ms.sc_full + sc.idx, sc.phase);
                if (!__all_sync(0xffffffffu, s_here && sc_here)) {
                    wait_warp(ms.sc_full + sc.idx, sc.phase);
                    wait_warp(ms.s_full + buf, (s_phase >> buf) & 1u);
                }
                tc_fence_after();
                s_phase ^= 1u << buf;
                // the keys' scales of 4 of this thread's 8 groups, times the row's; above 0, so that a score that is masked
                // by -inf stays so where the keys' scale is 0
                auto key_scales = [&](int k, float (&f)[4]) {
                    const float4 a = *reinterpret_cast<const float4*>(&ms.k_scale[sc.idx][half * 8 + k * 4]);
                    f[0] = fmaxf(a.x * c, 1e-30f), f[1] = fmaxf(a.y * c, 1e-30f);
                    f[2] = fmaxf(a.z * c, 1e-30f), f[3] = fmaxf(a.w * c, 1e-30f);
                };
                uint32_t r[2][32];
                float mx = -INFINITY;
                if (ok && busy) {
                    tmem_ld32(s_addr + half * 64, r[0]);
                    tmem_ld32(s_addr + half * 64 + 32, r[1]);
                    tmem_ld_wait();
                    reg_fence32(r[0]);
                    reg_fence32(r[1]);
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // keys kb .. kb + 31 that this row sees
                            const int32_t kb = key0 + half * 64 + 32 * k, a = kb - ctx;
                            uint32_t bits = 0u;
                            if (live_row) {
                                bits = bit_span(lo_s[nd] - kb, ctx - kb);
                                if (a > -32 && a < 0) {
                                    bits |= anc[0] << -a;
                                } else if (a >= 0 && a < pc.n) {
                                    const int wd = a >> 5;
                                    bits |= __funnelshift_r(anc[wd], wd + 1 < words ? anc[wd + 1] : 0u, a & 31);
                                }
                            }
#pragma unroll
                            for (int u = 0; u < 32; ++u) r[k][u] = (bits >> u) & 1u ? r[k][u] : 0xFF800000u;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float ksc[4];
                        key_scales(k, ksc);
                        const float4 v = *reinterpret_cast<const float4*>(&ms.v_log[sc.idx][half * 8 + k * 4]);
                        const float vlg[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint32_t* q = &r[k][g * 8];
                            float a = fmaxf(fmaxf(u2f(q[0]), u2f(q[1])), u2f(q[2]));
                            const float b = fmaxf(fmaxf(u2f(q[3]), u2f(q[4])), u2f(q[5]));
                            a = fmaxf(fmaxf(a, u2f(q[6])), u2f(q[7]));
                            mx = fmaxf(mx, fmaf(fmaxf(a, b), ksc[g], vlg[g]));
                        }
                    }
                }
                // Both halves of the row: its maximum, and S is read, so that P may take its place.
                sm.mx[buf][half][row] = mx;
                tc_fence_before();
                named_bar_sync_256();
                tc_fence_after();
                mx = fmaxf(mx, sm.mx[buf][half ^ 1][row]);
                const bool grow = live_row && mx > m2 + kRescaleThresh;
                float alpha = 1.f;
                if (grow) {
                    alpha = ex2(m2 - mx);  // 0 from -inf
                    m2 = mx;
                    l *= alpha;
                }
                // O holds the tiles before this one once their product is done: only a rescale waits for it here
                const bool rescale = t > 0 && __any_sync(0xffffffffu, grow);
                if (rescale) {
                    wait_warp(ms.p_free + (buf ^ 1), (o_phase >> (buf ^ 1)) & 1u);
                    if (ok) {
#pragma unroll 1
                        for (int32_t col = d0; col < d1; col += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_addr + col, o);
                            tmem_ld_wait();
                            reg_fence16(o);
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = f2u(u2f(o[u]) * alpha);
                            tmem_st16(o_addr + col, o);
                        }
                        tmem_st_wait();
                    }
                }
                if (half == 1) arrive(ms.p_half + buf);  // its part of O is rescaled
                if (ok && busy) {
                    const float mu = (m2 == -INFINITY ? 0.f : m2) - kLift + not_a_row;
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float ksc[4];
                        key_scales(k, ksc);
                        const float4 v = *reinterpret_cast<const float4*>(&ms.v_log[sc.idx][half * 8 + k * 4]);
                        const float4 n = *reinterpret_cast<const float4*>(&ms.v_inv[sc.idx][half * 8 + k * 4]);
                        const float vlg[4] = {v.x, v.y, v.z, v.w}, vin[4] = {n.x, n.y, n.z, n.w};
                        uint32_t pk[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            const int g = u / 4;
                            const float shift = vlg[g] - mu;
                            float a, b;
                            unpack2(fma2(pack2(u2f(r[k][2 * u]), u2f(r[k][2 * u + 1])), pack2(ksc[g], ksc[g]),
                                         pack2(shift, shift)), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[u & 1] = fma2(pack2(a, b), pack2(vin[g], vin[g]), sum[u & 1]);
                            const __half2 h2 = __floats2half2_rn(a, b);
                            pk[u] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        tmem_st16(s_addr + half * 32 + k * 16, pk);
                    }
                    float a, b;
                    unpack2(add2(sum[0], sum[1]), a, b);
                    l += a + b;
                    tmem_st_wait();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(ms.sc_free + sc.idx);
                sc.advance(1, kScaleRing);
                if (t > 0) o_phase ^= 1u << (buf ^ 1);  // (the phase of the tile before; never two behind)
                arrive((half == 0 ? ms.p_half : ms.p_full) + buf);
            }
            wait_warp(ms.p_free + ((steps - 1) & 1), (o_phase >> ((steps - 1) & 1)) & 1u);
            o_phase ^= 1u << ((steps - 1) & 1);
            // ---------------------------------------------------------------- output
            const bool whole = pc.whole != 0;
            const int64_t prow = tree_part_row(p, range, sub, pc.slot) + row;
            const int32_t node = node0 + nd, head = pc.g * p.G + st.gc * p.Gc + (row - nd * p.Gc);
            const int64_t orow = ((int64_t)pc.b * p.T + node) * p.Hq + head;
            tc_fence_before();
            sm.l[half][row] = l;
            named_bar_sync_256();
            tc_fence_after();
            const float tot = sm.l[0][row] + sm.l[1][row];
            const float inv = tree_inv_sum(tot, whole) * ms.v_ref;
            if (live_row && half == 0) {
                const float lse = tree_row_lse((m2 - kLift + log2f(tot)) * kLn2, tot, whole);
                if (!whole)
                    p.part_lse[prow] = lse;
                else if (p.lse)
                    p.lse[orow] = lse;
            }
            // each thread writes half of the row's columns
            if (ok && busy) {
#pragma unroll 1
                for (int32_t col = d0; col < d1; col += 16) {
                    uint32_t q[16];
                    tmem_ld16(o_addr + col, q);
                    tmem_ld_wait();
                    reg_fence16(q);
                    float o[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = u2f(q[u]) * inv;
                    if (live_row && !whole) {
                        float* dst = p.part_out + prow * DV + col;
                        store_f8(dst, o);
                        store_f8(dst + 8, o + 8);
                    } else if (live_row) {
                        uint32_t pk[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(o[2 * u], o[2 * u + 1]);
                            pk[u] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        uint4* dst =
                            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * p.D + col);
                        dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
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
            produce(p, x, w, node0, ms, &tm_v, r_ring, ms.r_full, ms.r_empty, x.r_stages, wait_all);
        } else if (warp == kScaleWarp) {
            fetch_scales(p, x, w, node0, ms, wait_all);
        } else if (warp >= kConvertWarp) {
            convert<kVN, DV>(p, x, w, st, node0, ms, q_s, r_ring, v_ring, wait_all);
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------------ MMA issuer: one thread
            constexpr uint32_t idesc_s = idesc_f8(128, kTile, 0, 0, 0);
            constexpr uint32_t idesc_o = idesc_f16(128, kVN, 0, 1);
            const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024), k_desc = sw128_desc(smem_u32(k_ring), 16, 1024),
                           v_desc = sw128_desc(smem_u32(v_ring), 8192, 1024);
            const uint32_t q_chunk = q_chunk_bytes / 16;  // hi, then lo of a chunk
            RingPos kp{0, 0u}, vp{0, 0u};
            uint32_t q_phase = 0, p_phase = 0;  // p_phase: bit b = parity of the next P in buffer b
            auto issue = [&](const Piece& pc) {
                const int32_t steps = pc.tiles;
                ok = wait_one(&ms.q_full, q_phase);
                if (!ok) return;
                q_phase ^= 1u;
                auto scores = [&](int32_t t) {
                    const uint32_t d = tmem + (uint32_t)(t & 1) * 128;
                    uint64_t qd = q_desc;
#pragma unroll 1
                    for (int32_t kc = 0; kc < kc_n; ++kc) {
                        ok = wait_one(ms.k_full + kp.idx, kp.phase);
                        if (!ok) return;
                        const uint64_t kd = k_desc + (uint32_t)kp.idx * (kStageBytes / 16);
                        const int32_t part = (min(128, p.D - kc * 128) + 31) / 32;  // steps of 32 dims; the rest is zeros
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk < part) {
                                tc_mma_f8(d, qd + 2 * kk, kd + 2 * kk, idesc_s, (kc > 0 || kk > 0) ? 1u : 0u);
                                tc_mma_f8(d, qd + q_chunk + 2 * kk, kd + 2 * kk, idesc_s, 1u);
                            }
                        }
                        tc_commit(ms.k_empty + kp.idx);
                        qd += 2 * q_chunk;
                        kp.advance(1, x.k_stages);
                    }
                    tc_commit(ms.s_full + (t & 1));
                    if (t == steps - 1) tc_commit(&ms.q_free);
                };
                auto values = [&](int32_t t) {
                    const uint32_t pa = tmem + (uint32_t)(t & 1) * 128;
                    // the first 64 keys' probabilities come ahead of the rest
                    ok = wait_one(ms.p_half + (t & 1), (p_phase >> (t & 1)) & 1u);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll 1
                    for (int32_t sv = 0; sv < kc_n * (kTile / kVKeys); ++sv) {
                        const int32_t c = sv / (kTile / kVKeys), h = sv - c * (kTile / kVKeys);
                        if (h == 1 && c == 0) {
                            ok = wait_one(ms.p_full + (t & 1), (p_phase >> (t & 1)) & 1u);
                            if (!ok) return;
                            tc_fence_after();
                        }
                        ok = wait_one(ms.v_full + vp.idx, vp.phase);
                        if (!ok) return;
                        const uint64_t vd = v_desc + (uint32_t)vp.idx * (kStageBytes / 16);
                        const uint32_t dc = tmem + kOCol + (uint32_t)c * 128, ph = pa + (uint32_t)(h * kVKeys) / 2;
                        auto part = [&](int k0) {
#pragma unroll
                            for (int kk = k0; kk < k0 + 4; ++kk)
                                tc_mma_ta(dc, ph + kk * 8, vd + kk * 128, idesc_o, (t > 0 || h > 0 || kk > 0) ? 1u : 0u);
                            };
                        part(0);
                        if (kVKeys == 128) {
                            ok = wait_one(ms.p_full + (t & 1), (p_phase >> (t & 1)) & 1u);
                            if (!ok) return;
                            tc_fence_after();
                            part(4);
                        }
                        tc_commit(ms.v_empty + vp.idx);
                        vp.advance(1, x.v_stages);
                    }
                    p_phase ^= 1u << (t & 1);
                    tc_commit(ms.p_free + (t & 1));
                };
                scores(0);
                if (ok && steps > 1) scores(1);
#pragma unroll 1
                for (int32_t t = 0; t < steps && ok; ++t) {
                    values(t);
                    if (ok && t + 2 < steps) scores(t + 2);
                }
            };
            each_piece(p, w, node0, ms, false, [&](const Piece& pc) {
                if (elect_one() && ok) issue(pc);
                __syncwarp();
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

// ------------------------------------------------------------------------------- host side

template <int DV>
cudaError_t launch_dv(const CUtensorMap& tk, const CUtensorMap& tv, const TreeAttnParams& p, Shape x, cudaStream_t stream)
{
    const int32_t q_bytes = 2 * ((p.D + 127) / 128) * x.q_rows * 128;
    const int32_t misc = (int32_t)sizeof(TcMisc) + p.npt * 4 * (1 + (p.T + 31) / 32);
    // (Q's 128-row reads past its last row end inside the rings)
    if (!deal_stages(x, kSmemMax - 1024 - q_bytes - misc)) return cudaErrorInvalidConfiguration;
    cudaError_t e =
        cudaFuncSetAttribute(cache8_attn_tc_kernel<DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.ranges * p.n_sub));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + q_bytes + (x.k_stages + x.r_stages + x.v_stages) * kStageBytes + misc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];  // set-up beside the end of the kernel before
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache8_attn_tc_kernel<DV>, tk, tv, p, x);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

}  // namespace

bool tc8::encode_maps(const TreeAttnParams& p, int32_t box, CUtensorMap* tk, CUtensorMap* tv)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    // a stride that is never taken (one head, one page) may be anything: the tensor map wants a plain one
    const int64_t sh = p.Hkv > 1 ? p.sh : p.D, sp = p.num_pages > 1 ? p.sp : p.ss * p.page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv, (cuuint64_t)p.page_size, (cuuint64_t)p.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)sh, (cuuint64_t)p.ss, (cuuint64_t)sp};
    const cuuint32_t shape[4] = {128, 1, (cuuint32_t)box, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    auto one = [&](CUtensorMap* map, const void* base) {
        return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, shape, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   p.D > 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return one(tk, p.k) && one(tv, p.v);
}

bool cache8_tc_supports(const dflash_dims* d)
{
    const int64_t most = int64_t(1) << 40;  // bytes: where a tensor map's strides end
    if (d->dtype != DFLASH_BF16) return false;
    if (d->kv_stride_slot <= 0 || (d->num_kv_heads > 1 && d->kv_stride_head <= 0) ||
        (d->num_pages > 1 && d->kv_stride_page <= 0))
        return false;
    return d->kv_stride_slot < most && d->kv_stride_head < most && d->kv_stride_page < most;
}

cudaError_t launch_cache8_attn_tc(const TreeAttnParams& p, cudaStream_t stream)
{
    Shape x{};
    x.q_rows = p.few ? (p.rows + 15) / 16 * 16 : (p.rows + 7) / 8 * 8;
    x.box = 8;
    while (x.box < 128 && p.page_size % (2 * x.box) == 0) x.box *= 2;
    const uint32_t groups = (uint32_t)p.page_size / kGroup;  // of a page
    x.page_magic = groups == 1 ? 0u : (uint32_t)(((1ull << 32) + groups - 1) / groups);
    CUtensorMap tk, tv;
    if (!tc8::encode_maps(p, x.box, &tk, &tv)) return cudaErrorNotSupported;
    if (p.few) return tc8::launch_few(tk, tv, p, x, stream);
    switch (p.DV) {
    case 64: return launch_dv<64>(tk, tv, p, x, stream);
    case 128: return launch_dv<128>(tk, tv, p, x, stream);
    default: return launch_dv<256>(tk, tv, p, x, stream);
    }
}

}  // namespace dflash
