// Tree attention on the tensor cores (bf16): tcgen05.mma with the scores, the probabilities and the output in
// TMEM, paged K/V staged by TMA into a shared-memory ring.
//
//   S [128 rows x 128 keys] = Q [128 x D] . K^T        (A: Q in shared memory, B: the K tile)
//   O [128 rows x DV]      += P [128 x 128] . V        (A: P in TMEM, B: the V tile, MN-major)
//
// A query row is a (node, head of the KV head's group), a TMEM lane. Two softmax threads share a row's tile, 64
// keys each: they read their scores once into registers, exchange one maximum through shared memory, and hand
// over their half of P. (A thread per row, alternate tiles to two warpgroups and O accumulators, took 1.45 us a
// tile, two passes over TMEM, on the way between two MMAs: 158 us for the ragged batch of 64-node trees.) P
// (bf16) overwrites its own S, thus costs neither shared memory nor TMEM, and shared memory is left to Q and
// the ring: what bounds the kernel is the K/V stream, whose rate is the bytes in flight over the latency.
//
// TMEM (512 columns): S0, S1 (128 each) and up to 256 of O; for head_dim above 256 a CTA computes 256 of the
// output's dims from the whole S. A query tile is up to 128 rows; step t of a piece (one range's part of a
// request and KV head) is its key tile t, with S buffer t % 2. The MMA warp does: S(0), S(1), then for every t:
// O += P(t) V, S(t + 2), which reuses the buffer of P(t) (MMAs of one thread execute in order), so S(t + 1)
// waits for the softmax while S(t)'s P is multiplied.
//
// More than 128 rows per KV head: CTA pairs (clusters of two, cta_group::2). The two CTAs hold neighbouring
// query tiles and share every MMA (M = 256): each loads half of the K tile's keys and half of the V tile's
// dims, so a K/V byte enters one SM for 256 rows, and an SM reads half of each B operand from its shared
// memory, which is what bounds an MMA of 128 x 128 x 16 (97 cycles measured with both operands in one SM's
// shared memory, against 64 at the tensor peak). The even CTA's thread issues; its commits arrive in both CTAs;
// softmax warps of both arrive at the even CTA's barriers. (Two tiles of 128 rows in one CTA instead took 177
// us for the ragged batch of 64-node trees, 2.6 us a tile of 128 keys, of which the MMAs were 1.5.)
//
// Online softmax about a lazy maximum: a row's maximum moves only when a score exceeds it by 2^8 in the exp2
// domain; O and the sum are then rescaled in place. P <= 2^8 in bf16 rounds each probability to 2^-8 relative,
// the same choice the block attention makes: the products with V average such errors out, and P in fp32 would
// need tf32 MMAs of a quarter of the rate. The row sums add the unrounded probabilities in fp32.
//
// Masks are only looked at in tiles that hold tree keys or a window's edge: a node's visible keys of 32
// positions are one word, made from its ancestors' bits. V rows that no node sees are zeroed in shared memory,
// as 0 x NaN would reach every row.
//
// Warps: 0-7 softmax and output, 8-10 TMA producers, 11 the MMA issuer. Ring stages are 16 KB: K 128 keys x 64
// dims, V 64 keys x 128 dims (128 keys x 64 dims at DV = 64); in a pair each CTA's halves are K 64 keys x 128
// dims, V 64 keys x 128 dims (DV = 256) or 128 keys x 64 dims. A box is 64 dims of up to 64 tokens of one page;
// its id is read one stage ahead by the lane that issues it. Boxes past the keys or before the window are
// fetched at an out-of-bounds page, which the TMA unit fills with zeros without a look at the table.
//
// Bounds and what was measured (calls back to back, ranges over several GPUs): long contexts the K/V stream, 4
// requests of 120k to 128k keys, 32 nodes, 32/8 heads of 128: 324 to 342 us, 6.0 to 6.35 TB/s. Many rows per key
// the chain MMA - softmax - MMA, 8 ragged requests of up to 32k keys, 64 nodes: 133 to 138 us, 0.93 to 0.96 PFLOP/s
// (0.85 us a pair tile, of which the MMAs are some 0.65). Short calls the start (lengths, page table, first K: 6 us),
// the bytes an SM takes in (some 44 GB/s of the whole rate each) and the join: one request of 8192 keys, 24 nodes,
// 32/4 heads of 512: 33 us; 4 sliding windows of 1024, 16 nodes, 32/16 heads of 256: 28 us.
//
// Every mbarrier wait is bounded (p.wait_ns): on expiry the kernel records DFLASH_DEVERR_TIMEOUT, waits
// (bounded) for its own copies and MMAs, frees TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace dflash {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kSoftmax = 256;  // warps 0-7
constexpr int kProducerWarp = 8;
constexpr int kProducers = 3;
constexpr int kMmaWarp = 11;
constexpr int kTile = 128;
constexpr int kStageBytes = 16384;
constexpr int kMaxStages = 13;
constexpr int kSmemMax = 227 * 1024;
constexpr int kOCol = 256;  // first TMEM column of O
// After a failed wait, whatever the caller's limit: the bound of the waits for copies and MMAs in flight, and
// the time given to copies that this CTA cannot wait for.
constexpr unsigned long long kDrainNs = 100000000ull;
constexpr unsigned long long kCopyGraceNs = 1000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThresh = 8.0f;

struct TcShape {
    int32_t stages;   // ring depth
    int32_t q_rows;   // rows of Q in shared memory (p.rows rounded up to 8)
    int32_t box;      // tokens per box
};

// Shared memory after the alignment gap: Q, the ring, then this.
struct TcMisc {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full, q_free;
    uint64_t s_full[2], p_half[2], p_full[2], o_done;
    uint64_t v_clean[kMaxStages];  // pair: the odd CTA has zeroed its rows of the slot's V stage
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
    float mx[2][2][128];  // row maxima of tile t over half of its keys, in [t % 2]
    float l[2][128];
    int32_t par[DFLASH_MAX_TREE_NODES];
    // then lo [npt], ancestor words [npt][(T + 31) / 32]
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Orders later uses of loaded registers after the wait for the loads.
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32])
{
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 bytes, a whole sector, in one store.
__device__ __forceinline__ void store_f8(float* dst, const float* v)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// D (TMEM) (+)= A (TMEM, bf16 pairs) . B (shared memory)
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
        : "memory");
}

__device__ __forceinline__ void tc_mma2_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
        : "memory");
}

// Arrives on a barrier of another CTA of the cluster.
__device__ __forceinline__ void arrive_peer(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// One thread of the warp, always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// A ring position that advances by `by` stages.
struct RingPos {
    int32_t idx;
    uint32_t phase;
    __device__ __forceinline__ void advance(int by, int stages)
    {
        idx += by;
        if (idx >= stages) {
            idx -= stages;
            phase ^= 1u;
        }
    }
};

// What ring stage i of a piece of n tiles holds: K0 K1 V0 K2 V1 ... V(n-1), ks stages of a K tile and vs of a V tile.
struct StageOf {
    bool is_k;
    int32_t tile, sub;
};

__device__ __forceinline__ StageOf stage_of(int32_t i, int32_t n, int32_t ks, int32_t vs)
{
    if (i < ks) return StageOf{true, 0, i};
    const int32_t j = (i - ks) / (ks + vs), r = i - ks - j * (ks + vs);
    const bool is_k = j < n - 1 && r < ks;
    return StageOf{is_k, is_k ? j + 1 : j, is_k || j == n - 1 ? r : r - ks};
}

// Bits a .. b - 1 of a word (a and b outside [0, 32] are taken to its ends).
__device__ __forceinline__ uint32_t bit_span(int32_t a, int32_t b)
{
    a = max(a, 0);
    b = min(b, 32);
    if (b <= a) return 0u;
    return (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

template <int DV, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const TreeAttnParams p, const TcShape x)
{
    static_assert(DV == 256 || DV == 128 || (DV == 64 && !kPair), "64 dims in halves of 32 have no 128-byte rows");
    constexpr int kVN = kPair ? DV : DV == 64 ? 64 : 128;             // dims of a V stage (both CTAs' of a pair)
    constexpr int kVKeys = kPair ? (DV == 256 ? 64 : 128) : DV == 64 ? 128 : 64;  // and its keys
    constexpr int kM = kPair ? 256 : 128;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int32_t kc_n = (p.D + 63) / 64;
    uint8_t* q_s = smem;
    uint8_t* ring = smem + (size_t)kc_n * x.q_rows * 128;
    TcMisc& ms = *reinterpret_cast<TcMisc*>(ring + (size_t)x.stages * kStageBytes);
    int32_t* lo_s = reinterpret_cast<int32_t*>(&ms + 1);
    uint32_t* anc_s = reinterpret_cast<uint32_t*>(lo_s + p.npt);
    volatile int* abort_flag = &ms.abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int32_t range = blockIdx.x / p.n_sub, sub = blockIdx.x % p.n_sub;
    const SubTile st = sub_tile(p, sub);
    const int32_t node0 = st.rt * p.npt;
    const int32_t lead0 = (st.rt - (int32_t)rank) * p.npt;  // the even CTA's first node
    const int32_t ks_n = kPair ? (kc_n + 1) / 2 : kc_n;     // K stages per tile
    const int32_t vc_n = kPair ? 1 : (min(DV, p.D - st.dv * DV) + kVN - 1) / kVN;  // V column groups
    const int32_t vs_n = (kTile / kVKeys) * vc_n;                                   // V stages per tile
    const int S = x.stages;

    // What the barriers hand over lies in TMEM (ordered by the tcgen05 fences) or came by the async proxy: waits and
    // arrivals need no cluster-scope ordering of ordinary memory, which cost a softmax warp about 1 us per arrival.
    auto bounded_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return ring_wait(bar, parity, abort_flag, p.err, p.wait_ns);
    };
    // the even CTA's copy of a barrier
    auto lead_bar = [&](uint64_t* bar) -> uint32_t { return mapa_shared(smem_u32(bar), 0); };
    auto commit = [&](uint64_t* bar) {
        if (kPair)
            tc_commit2_both(bar);
        else
            tc_commit(bar);
    };

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(ms.full + i, 1);
            mbar_init(ms.empty + i, 1);
            mbar_init(ms.v_clean + i, 1);
        }
        mbar_init(&ms.q_full, 1);
        mbar_init(&ms.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(ms.s_full + i, 1);
            mbar_init(ms.p_half + i, kPair ? 16 : 8);  // a softmax warp each
            mbar_init(ms.p_full + i, kPair ? 8 : 4);
        }
        mbar_init(&ms.o_done, 1);
        mbar_init(&ms.drain, 1);
        ms.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if (kPair) {
            tmem_alloc2(&ms.tmem, 512);
            tmem_relinquish2();
        } else {
            tmem_alloc(&ms.tmem, 512);
            tmem_relinquish();
        }
    }
    cudaGridDependencySynchronize();  // the kernel before may still run until here
    PieceWalk w;
    w.start(p, range);
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync_all();  // the peer's barriers are set up before anything arrives there
    tc_fence_after();
    cudaTriggerProgrammaticLaunchCompletion();  // the join grid may take its place; it waits for this one to end
    const uint32_t tmem = ms.tmem;
    bool ok = true;
    // (the odd CTA of a pair may have no row of its own, but shares the work on the even one's)
    auto skip = [&]() -> bool { return w.req.n <= lead0; };
    // a tile with V rows that no node sees
    auto edge_of = [&](int32_t tile) -> bool {
        const int32_t key0 = (w.req.tile0 + w.t0 + tile) * kTile;
        return key0 < w.req.lo || key0 + kTile > w.req.L;
    };
    // Zeroes those rows of a V stage (its keys begin at key0); 0 x NaN would reach every row. Boxes without a visible
    // key came as zeros, so only the rest of the two boxes at the edges is left.
    auto clean = [&](uint8_t* stg, int32_t key0) {
        auto zero = [&](int32_t from, int32_t to) {
            const int32_t r0 = max(from - key0, 0), rows = min(to - key0, kVKeys) - r0;
            const int32_t slabs = kStageBytes / (kVKeys * 128);
            for (int32_t idx = lane; idx < rows * 8 * slabs; idx += 32) {
                const int32_t slab = idx / (rows * 8), rest = idx - slab * rows * 8;
                *reinterpret_cast<uint4*>(stg + slab * (kVKeys * 128) + (r0 + (rest >> 3)) * 128 + (rest & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
        };
        zero(w.req.lo & ~(x.box - 1), w.req.lo);
        zero(w.req.L, (w.req.L + x.box - 1) & ~(x.box - 1));
        fence_proxy_async_smem();
        __syncwarp();
    };

    if (warp >= kProducerWarp && warp < kProducerWarp + kProducers) {
        // ------------------------------------------------------------------ TMA producers
        const int pw = warp - kProducerWarp;
        const uint64_t kv_policy = l2_policy_evict_first();
        const int32_t boxes = kTile / x.box;  // per stage, K and V alike
        const bool once = p.n_sub == (kPair ? 2 : 1);
        RingPos pos{pw, 0u};
        uint32_t issued = 0, issued_phase = 0, q_phase = 0;
        bool q_out = false;
        int32_t skew = pw;  // this warp's next stage of the piece: every third one, counted across pieces
        for (; !w.done() && ok; w.next(p)) {
            if (skip()) continue;
            const int32_t n = w.t1 - w.t0;
            const int32_t total = n * (ks_n + vs_n);
            if (pw == 0) {
                // Q once the last piece's scores are computed
                ok = __all_sync(0xffffffffu, bounded_wait(&ms.q_free, q_phase ^ 1u));
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t bytes = (uint32_t)(kc_n * p.rows * 128);
                    if (leader) mbar_expect_tx(&ms.q_full, kPair ? 2 * bytes : bytes);
                    for (int kc = 0; kc < kc_n; ++kc) {
                        uint8_t* dst = q_s + (size_t)kc * x.q_rows * 128;
                        const int32_t head = w.g * p.G + st.gc * p.Gc;
                        if (kPair)
                            tma_load_3d_pair(dst, &tm_q, lead_bar(&ms.q_full), kc * 64, head, w.b * p.T + node0);
                        else
                            tma_load_3d(dst, &tm_q, &ms.q_full, kc * 64, head, w.b * p.T + node0);
                    }
                }
                __syncwarp();
                q_phase ^= 1u;
                q_out = true;
            }
            // this lane's box of stage i: page id and coordinates
            struct Box {
                int32_t page, slot, dim, dst;
            };
            auto box_of = [&](int32_t i) -> Box {
                Box bx{p.num_pages, 0, 0, 0};
                if (lane >= boxes) return bx;
                const StageOf so = stage_of(i, n, ks_n, vs_n);
                int32_t key = (w.req.tile0 + w.t0 + so.tile) * kTile;
                const int32_t per = boxes / 2, slab = lane / per, i2 = lane - slab * per;  // of two 64-dim slabs
                bool slabs;
                if (so.is_k) {
                    slabs = kPair;
                    key += kPair ? (int32_t)rank * 64 : 0;
                    bx.dim = so.sub * (kPair ? 128 : 64);
                } else {
                    slabs = kVKeys == 64;
                    const int32_t h = so.sub / vc_n, c = so.sub - h * vc_n;
                    key += h * kVKeys;
                    bx.dim = st.dv * DV + c * kVN + (int32_t)rank * (kVN / 2);
                }
                if (slabs) {
                    key += i2 * x.box;
                    bx.dim += slab * 64;
                    bx.dst = slab * 8192 + i2 * x.box * 128;
                } else {
                    key += lane * x.box;
                    bx.dst = lane * x.box * 128;
                }
                if (key < w.req.L && key + x.box > w.req.lo) {
                    const int32_t pg = key / p.page_size;
                    bx.slot = key - pg * p.page_size;
                    const int32_t id = __ldg(p.page_table + (int64_t)w.b * p.max_pages + pg);
                    if (id >= 0 && id < p.num_pages)
                        bx.page = id;
                    else
                        raise_error(p.err, DFLASH_DEVERR_PAGE_ID);
                }
                return bx;
            };
            int32_t i = skew;
            Box cur{p.num_pages, 0, 0, 0};
            if (i < total) cur = box_of(i);
#pragma unroll 1
            for (; i < total; i += kProducers) {
                Box nxt{p.num_pages, 0, 0, 0};
                if (i + kProducers < total) nxt = box_of(i + kProducers);
                ok = __all_sync(0xffffffffu, bounded_wait(ms.empty + pos.idx, pos.phase ^ 1u));
                if (!ok) break;
                const StageOf so = stage_of(i, n, ks_n, vs_n);
                // Pair: the even CTA's barrier counts both halves of a stage; but where V rows have to be zeroed
                // each CTA's counts its own, and the odd one reports when it has done so (v_clean).
                const bool apart = kPair && !so.is_k && edge_of(so.tile);
                if (lane == 0 && (leader || apart))
                    mbar_expect_tx(ms.full + pos.idx, kPair && !apart ? 2 * kStageBytes : kStageBytes);
                __syncwarp();
                if (lane < boxes) {
                    const CUtensorMap* map = so.is_k ? &tm_k : &tm_v;
                    uint8_t* dst = ring + (size_t)pos.idx * kStageBytes + cur.dst;
                    // read once: the first to leave L2, unless other query tiles read it again
                    if (kPair) {
                        const uint32_t bar = mapa_shared(smem_u32(ms.full + pos.idx), apart ? rank : 0u);
                        if (once)
                            tma_load_4d_pair_hint(dst, map, bar, cur.dim, w.g, cur.slot, cur.page, kv_policy);
                        else
                            tma_load_4d_pair(dst, map, bar, cur.dim, w.g, cur.slot, cur.page);
                    } else if (once) {
                        tma_load_4d_hint(dst, map, ms.full + pos.idx, cur.dim, w.g, cur.slot, cur.page, kv_policy);
                    } else {
                        tma_load_4d(dst, map, ms.full + pos.idx, cur.dim, w.g, cur.slot, cur.page);
                    }
                }
                __syncwarp();
                issued |= 1u << pos.idx;
                issued_phase = (issued_phase & ~(1u << pos.idx)) | (pos.phase << pos.idx);
                pos.advance(kProducers, S);
                cur = nxt;
            }
            skew = i - total;
        }
        // No copy of ours may land after the CTA has gone. The odd CTA's are counted at the even one's barriers, which
        // it cannot wait on: it gives them time.
        if (!ok && lane == 0) {
            const unsigned long long t0 = globaltimer();
            if (leader) {
                for (int s = 0; s < S; ++s)
                    if (issued & (1u << s))
                        while (!mbar_test_wait(ms.full + s, (issued_phase >> s) & 1u) && globaltimer() - t0 < kDrainNs) {
                        }
                if (q_out)
                    while (!mbar_test_wait(&ms.q_full, q_phase ^ 1u) && globaltimer() - t0 < kDrainNs) {
                    }
            }
            if (kPair)
                while (globaltimer() - t0 < kCopyGraceNs) {
                }
        }
        __syncwarp();
    } else if (warp == kMmaWarp && leader) {
        // ------------------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc_s = make_idesc(kM, kTile, 0, 0);
        constexpr uint32_t idesc_o = make_idesc(kM, kVN, 0, 1);
        // Descriptors are made once: a later operand is its base plus an offset in 16-byte units. Everything about an
        // MMA but the issue itself is the same for the whole warp, so that it lies in uniform registers, where the
        // instruction wants it; with the operands worked out by one thread an MMA took about 150 cycles to issue.
        const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024), k_desc = sw128_desc(smem_u32(ring), 16, 1024),
                       v_desc = sw128_desc(smem_u32(ring), 8192, 1024);
        const uint32_t q_chunk = (uint32_t)x.q_rows * 8;  // one 64-dim chunk of Q
        RingPos pos{0, 0u};
        // p_phase: bit b = parity of the next P in buffer b; clean_phase: bit s = of slot s's next zeroed V stage
        uint32_t q_phase = 0, p_phase = 0, clean_phase = 0;
        auto wait0 = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, bounded_wait(bar, parity));
        };
        for (; !w.done() && ok; w.next(p)) {
            if (skip()) continue;
            const int32_t steps = w.t1 - w.t0;
            ok = wait0(&ms.q_full, q_phase);
            if (!ok) break;
            q_phase ^= 1u;
            // S(t) = Q K^T
            auto scores = [&](int32_t t) {
                const uint32_t d = tmem + (uint32_t)(t & 1) * 128;
                uint64_t qd = q_desc;
#pragma unroll 1
                for (int ks = 0; ks < ks_n; ++ks) {
                    ok = wait0(ms.full + pos.idx, pos.phase);
                    if (!ok) return;
                    const uint64_t kd = k_desc + (uint32_t)pos.idx * (kStageBytes / 16);
                    const bool second = kPair && 2 * ks + 1 < kc_n;  // the stage's second slab holds dims
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kPair)
                                tc_mma2(d, qd + 2 * kk, kd + 2 * kk, idesc_s, (ks > 0 || kk > 0) ? 1u : 0u);
                            else
                                tc_mma(d, qd + 2 * kk, kd + 2 * kk, idesc_s, (ks > 0 || kk > 0) ? 1u : 0u);
                        }
                        if (second) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma2(d, qd + q_chunk + 2 * kk, kd + 512 + 2 * kk, idesc_s, 1u);
                        }
                        commit(ms.empty + pos.idx);
                    }
                    __syncwarp();
                    qd += kPair ? 2 * q_chunk : q_chunk;
                    pos.advance(1, S);
                }
                if (elect_one()) commit(ms.s_full + (t & 1));
                __syncwarp();
            };
            // O += P(t) V
            auto values = [&](int32_t t) {
                const bool first = t == 0;
                const uint32_t d = tmem + kOCol;
                const uint32_t pa = tmem + (uint32_t)(t & 1) * 128;
                const bool edge = edge_of(t);
                // the first 64 keys' probabilities come ahead of the rest
                ok = wait0(ms.p_half + (t & 1), (p_phase >> (t & 1)) & 1u);
                if (!ok) return;
                tc_fence_after();
#pragma unroll 1
                for (int sv = 0; sv < vs_n; ++sv) {
                    const int32_t h = sv / vc_n, c = sv - h * vc_n;
                    if (h == 1 && c == 0) {
                        ok = wait0(ms.p_full + (t & 1), (p_phase >> (t & 1)) & 1u);
                        if (!ok) return;
                        tc_fence_after();
                    }
                    ok = wait0(ms.full + pos.idx, pos.phase);
                    if (!ok) return;
                    if (edge) {
                        clean(ring + (size_t)pos.idx * kStageBytes, (w.req.tile0 + w.t0 + t) * kTile + h * kVKeys);
                        if (kPair) {
                            // (the odd CTA's ordinary stores come before its arrival)
                            ok = __all_sync(0xffffffffu,
                                            ring_wait_cluster(ms.v_clean + pos.idx, (clean_phase >> pos.idx) & 1u,
                                                              abort_flag, p.err, p.wait_ns));
                            if (!ok) return;
                            clean_phase ^= 1u << pos.idx;
                        }
                    }
                    const uint64_t vd = v_desc + (uint32_t)pos.idx * (kStageBytes / 16);
                    const uint32_t dc = d + (uint32_t)c * 128, ph = pa + (uint32_t)(h * kVKeys) / 2;
                    auto part = [&](int k0) {
                        if (elect_one()) {
#pragma unroll
                            for (int kk = k0; kk < k0 + 4; ++kk) {
                                const uint32_t more = (!first || h > 0 || kk > 0) ? 1u : 0u;
                                if (kPair)
                                    tc_mma2_ta(dc, ph + kk * 8, vd + kk * 128, idesc_o, more);
                                else
                                    tc_mma_ta(dc, ph + kk * 8, vd + kk * 128, idesc_o, more);
                            }
                        }
                        __syncwarp();
                    };
                    part(0);
                    if (kVKeys == 128) {
                        ok = wait0(ms.p_full + (t & 1), (p_phase >> (t & 1)) & 1u);
                        if (!ok) return;
                        tc_fence_after();
                        part(4);
                    }
                    if (elect_one()) commit(ms.empty + pos.idx);
                    __syncwarp();
                    pos.advance(1, S);
                }
                p_phase ^= 1u << (t & 1);
                if (elect_one()) commit(&ms.o_done);
                __syncwarp();
            };
            scores(0);
            if (ok && steps > 1) scores(1);
#pragma unroll 1
            for (int32_t t = 0; t < steps && ok; ++t) {
                values(t);
                if (ok && t + 2 < steps) scores(t + 2);
            }
            if (ok && elect_one()) commit(&ms.q_free);
            __syncwarp();
        }
        // our MMAs end before TMEM is freed
        if (elect_one()) {
            if (kPair)
                tc_commit2_local(&ms.drain);
            else
                tc_commit(&ms.drain);
            const unsigned long long t0 = globaltimer();
            while (!mbar_test_wait(&ms.drain, 0) && globaltimer() - t0 < kDrainNs) {
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------------ odd CTA: rows of V to zero
        RingPos pos{0, 0u};
        uint32_t seen = 0;  // bit s: parity of the next stage counted at this CTA's own full[s]
        for (; !w.done() && ok; w.next(p)) {
            if (skip()) continue;
            const int32_t n = w.t1 - w.t0;
            const int32_t total = n * (ks_n + vs_n);
#pragma unroll 1
            for (int32_t i = 0; i < total && ok; ++i, pos.advance(1, S)) {
                const StageOf so = stage_of(i, n, ks_n, vs_n);
                if (so.is_k || !edge_of(so.tile)) continue;
                ok = __all_sync(0xffffffffu, bounded_wait(ms.full + pos.idx, (seen >> pos.idx) & 1u));
                if (!ok) break;
                seen ^= 1u << pos.idx;
                clean(ring + (size_t)pos.idx * kStageBytes, (w.req.tile0 + w.t0 + so.tile) * kTile + so.sub * kVKeys);
                if (lane == 0) mbar_arrive_cluster(lead_bar(ms.v_clean + pos.idx));
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------------------------ softmax and output
        // Warps w and w + 4 share TMEM lanes, that is rows: a row's tile is split between two threads, of its first and
        // its last 64 keys.
        const int half = warp >> 2;
        const int row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float sl2 = p.scale * kLog2e;
        const int words = (p.T + 31) / 32;
        uint32_t s_phase = 0, o_phase = 0;  // s_phase: bit b = parity of the next S in buffer b
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, bounded_wait(bar, parity));
            tc_fence_after();
        };
        // a softmax warp's part of P is in TMEM
        auto arrive = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair && !leader)
                    arrive_peer(lead_bar(bar));
                else
                    mbar_arrive(bar);
            }
        };
        int32_t masks_of = -1;  // the request whose nodes' masks are in shared memory
        // A failed wait ends the computation, not the walk: the barriers below are met by every thread.
        for (; !w.done(); w.next(p)) {
            if (skip()) continue;
            const int32_t live = min(p.npt, w.req.n - node0) * p.Gc;  // rows of this CTA with a node; <= 0: none
            const int32_t steps = w.t1 - w.t0;
            const int32_t ctx = w.req.ctx;
            const int32_t first_key = (w.req.tile0 + w.t0) * kTile, end_key = (w.req.tile0 + w.t1) * kTile;
            const int32_t win_end = p.window > 0 ? ctx + w.req.n - p.window : 0;  // keys from here on: no window's edge
            if ((end_key > ctx || first_key < win_end) && masks_of != w.b) {
                masks_of = w.b;  // (the KV heads of a request share them)
                // (the barrier that ended the last piece keeps its masks from being overwritten)
                tree_load_parents(p, w.b, w.req.n, ms.par, tid, kSoftmax);
                named_bar_sync_256();
                tree_walk_nodes(p, w.req, node0, min(p.npt, w.req.n - node0), ms.par, anc_s, lo_s, tid,
                                kSoftmax);
                named_bar_sync_256();
            }
            const bool live_row = row < live;
            const int32_t nd = row / p.Gc;
            const uint32_t* anc = anc_s + nd * words;
            const uint32_t o_addr = tmem + kOCol + lanes;
            const int32_t d_here = min(DV, p.D - st.dv * DV);
            const int32_t d0 = half * (DV / 2), d1 = min(d_here, d0 + DV / 2);  // this thread's share of O's columns
            float m2 = -INFINITY, l = 0.f;  // the row's maximum, and the sum over this thread's keys
#pragma unroll 1
            for (int32_t t = 0; t < steps; ++t) {
                const int buf = t & 1;
                const int32_t key0 = first_key + t * kTile;
                const bool edge = key0 + kTile > ctx || key0 < win_end;
                const uint32_t s_addr = tmem + (uint32_t)buf * 128 + lanes;
                wait_warp(ms.s_full + buf, (s_phase >> buf) & 1u);
                s_phase ^= 1u << buf;
                uint32_t r[2][32];
                float mx = -INFINITY;
                if (ok) {
                    tmem_ld32(s_addr + half * 64, r[0]);
                    tmem_ld32(s_addr + half * 64 + 32, r[1]);
                    tmem_ld_wait();
                    reg_fence32(r[0]);
                    reg_fence32(r[1]);
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // keys kb .. kb + 31 that this row sees
                            const int32_t kb = key0 + half * 64 + 32 * c, a = kb - ctx;
                            uint32_t bits = 0u;
                            if (live_row) {
                                bits = bit_span(lo_s[nd] - kb, ctx - kb);
                                if (a > -32 && a < 0) {
                                    bits |= anc[0] << -a;
                                } else if (a >= 0 && a < w.req.n) {
                                    const int wd = a >> 5;
                                    bits |= __funnelshift_r(anc[wd], wd + 1 < words ? anc[wd + 1] : 0u, a & 31);
                                }
                            }
#pragma unroll
                            for (int u = 0; u < 32; ++u) r[c][u] = (bits >> u) & 1u ? r[c][u] : 0xFF800000u;
                        }
                    }
                    float mc[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mc[i] = u2f(r[0][i]);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int u = c == 0 ? 4 : 0; u + 8 <= 32; u += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mc[i] = fmaxf(fmaxf(mc[i], u2f(r[c][u + i])), u2f(r[c][u + 4 + i]));
#pragma unroll
                    for (int i = 0; i < 4; ++i) mc[i] = fmaxf(mc[i], u2f(r[0][28 + i]));
                    mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
                }
                // Both halves of the row: its maximum, and S is read, so that P may take its place.
                ms.mx[buf][half][row] = mx;
                tc_fence_before();
                named_bar_sync_256();
                tc_fence_after();
                mx = fmaxf(mx, ms.mx[buf][half ^ 1][row]) * sl2;
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
                    wait_warp(&ms.o_done, o_phase);
                    if (ok) {
#pragma unroll 1
                        for (int32_t c = d0; c < d1; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_addr + c, o);
                            tmem_ld_wait();
                            reg_fence16(o);
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = f2u(u2f(o[u]) * alpha);
                            tmem_st16(o_addr + c, o);
                        }
                        tmem_st_wait();
                    }
                }
                if (half == 1) arrive(ms.p_half + buf);  // its part of O is rescaled
                if (ok) {
                    const float mu = m2 == -INFINITY ? 0.f : m2;
                    const uint64_t scale2 = pack2(sl2, sl2), shift2 = pack2(-mu, -mu);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            float a, b;
                            unpack2(fma2(pack2(u2f(r[c][2 * u]), u2f(r[c][2 * u + 1])), scale2, shift2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[u & 1] = add2(sum[u & 1], pack2(a, b));
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
                            pk[u] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        tmem_st16(s_addr + half * 32 + c * 16, pk);
                    }
                    float a, b;
                    unpack2(add2(sum[0], sum[1]), a, b);
                    l += a + b;
                    tmem_st_wait();
                }
                // (every phase of o_done is waited for once, so that its parity tells them apart)
                if (t > 0) {
                    if (!rescale) wait_warp(&ms.o_done, o_phase);
                    o_phase ^= 1u;
                }
                arrive((half == 0 ? ms.p_half : ms.p_full) + buf);
            }
            wait_warp(&ms.o_done, o_phase);
            o_phase ^= 1u;
            // ---------------------------------------------------------------- output
            const bool whole = w.whole();
            const int64_t prow = tree_part_row(p, range, sub, w.slot()) + row;
            const int32_t node = node0 + nd, head = w.g * p.G + st.gc * p.Gc + (row - nd * p.Gc);
            const int64_t orow = ((int64_t)w.b * p.T + node) * p.Hq + head;
            tc_fence_before();
            ms.l[half][row] = l;
            named_bar_sync_256();
            tc_fence_after();
            const float tot = ms.l[0][row] + ms.l[1][row];
            const float inv = tree_inv_sum(tot, whole);
            if (live_row && half == 0) {
                // (the sum of a row is 1 or more: __log2f is off by 2^-22 up to 2, by 2 ulp of the logarithm above)
                const float lse = tree_row_lse((m2 + __log2f(tot)) * kLn2, tot, whole);
                if (!whole)
                    p.part_lse[prow] = lse;
                else if (p.lse && st.dv == 0)
                    p.lse[orow] = lse;
            }
            // each thread writes half of the row's columns
            if (ok) {
#pragma unroll 1
                for (int32_t c = d0; c < d1; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(o_addr + c, r);
                    tmem_ld_wait();
                    reg_fence16(r);
                    float o[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = u2f(r[u]) * inv;
                    if (live_row && !whole) {
                        float* dst = p.part_out + prow * DV + c;
                        store_f8(dst, o);
                        store_f8(dst + 8, o + 8);
                    } else if (live_row) {
                        uint32_t pk[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(o[2 * u], o[2 * u + 1]);
                            pk[u] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * p.D +
                                                              st.dv * DV + c);
                        dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    }
                    __syncwarp();  // the next load takes the whole warp
                }
            }
            tc_fence_before();
            named_bar_sync_256();  // O, the sums and the masks are read before the next piece's steps
        }
    }
    // ---------------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync_all();  // no CTA leaves while the pair's MMAs or the peer may touch its memory
    if (warp == kMmaWarp) {
        tc_fence_after();
        if (kPair)
            tmem_dealloc2(tmem, 512);
        else
            tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------- host side

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

bool encode(EncodeTiledFn enc, CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box)
{
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_pairs_mutex;
int g_pairs[64][2] = {};  // resident CTA pairs per device, of DV = 128 and 256

// CTA pairs that are resident at once: a pair more would run after all the others.
template <int DV>
int resident_pairs()
{
    int dev = 0;
    const int guess = device_sm_count() / 2;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return guess;
    std::lock_guard<std::mutex> lk(g_pairs_mutex);
    int& n = g_pairs[dev][DV == 256];
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemMax;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int found = 0;
        if (cudaOccupancyMaxActiveClusters(&found, tree_attn_tc_kernel<DV, true>, &cfg) != cudaSuccess || found < 1) {
            (void)cudaGetLastError();
            return guess;
        }
        n = found;
    }
    return n;
}

template <int DV, bool kPair>
cudaError_t launch_dv(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, TreeAttnParams& p, int32_t box,
                      cudaStream_t stream)
{
    TcShape x;
    x.q_rows = (p.rows + 7) / 8 * 8;
    x.box = box;
    const int32_t q_bytes = (p.D + 63) / 64 * x.q_rows * 128;
    const int32_t misc = (int32_t)sizeof(TcMisc) + p.npt * 4 * (1 + (p.T + 31) / 32);
    x.stages = std::min(kMaxStages, (kSmemMax - 1024 - q_bytes - misc) / kStageBytes);
    // Q's 128-row reads past its last row end inside the ring
    if (x.stages < 4) return cudaErrorInvalidConfiguration;
    cudaError_t e =
        cudaFuncSetAttribute(tree_attn_tc_kernel<DV, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    if constexpr (kPair) p.ranges = std::max(1, std::min(p.ranges, 2 * resident_pairs<DV>() / p.n_sub));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.ranges * p.n_sub));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + q_bytes + x.stages * kStageBytes + misc;
    cfg.stream = stream;
    // set-up beside the end of the kernel before, a layer's join mostly: 8192 keys of 32/4 heads of 512, 35.4 -> 32.8 us a
    // call back to back
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, tree_attn_tc_kernel<DV, kPair>, tq, tk, tv, static_cast<const TreeAttnParams&>(p), x);
}

}  // namespace

bool tree_tc_supports(const dflash_dims* d)
{
    const int64_t most = int64_t(1) << 39;  // elements: a tensor map's strides end at 2^40 bytes
    if (d->dtype != DFLASH_BF16) return false;
    if (d->kv_stride_slot <= 0 || (d->num_kv_heads > 1 && d->kv_stride_head <= 0) ||
        (d->num_pages > 1 && d->kv_stride_page <= 0))
        return false;
    return d->kv_stride_slot < most && d->kv_stride_head < most && d->kv_stride_page < most;
}

cudaError_t launch_tree_attn_tc(TreeAttnParams& p, cudaStream_t stream)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    int32_t box = 8;
    while (box < 64 && p.page_size % (2 * box) == 0) box *= 2;
    CUtensorMap tq, tk, tv;
    const cuuint64_t qd[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hq, (cuuint64_t)p.B * p.T};
    const cuuint64_t qs[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.Hq * p.D * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)p.Gc, (cuuint32_t)p.npt};
    // a stride that is never taken (one head, one page) may be anything: the tensor map wants a plain one
    const int64_t sh = p.Hkv > 1 ? p.sh : p.D, sp = p.num_pages > 1 ? p.sp : p.ss * p.page_size;
    const cuuint64_t kd[4] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv, (cuuint64_t)p.page_size, (cuuint64_t)p.num_pages};
    const cuuint64_t ks[3] = {(cuuint64_t)sh * 2, (cuuint64_t)p.ss * 2, (cuuint64_t)sp * 2};
    const cuuint32_t kb[4] = {64, 1, (cuuint32_t)box, 1};
    if (!encode(enc, &tq, p.q, 3, qd, qs, qb) || !encode(enc, &tk, p.k, 4, kd, ks, kb) ||
        !encode(enc, &tv, p.v, 4, kd, ks, kb))
        return cudaErrorInvalidValue;
    if (p.pair)
        return p.DV == 128 ? launch_dv<128, true>(tq, tk, tv, p, box, stream)
                           : launch_dv<256, true>(tq, tk, tv, p, box, stream);
    switch (p.DV) {
    case 64: return launch_dv<64, false>(tq, tk, tv, p, box, stream);
    case 128: return launch_dv<128, false>(tq, tk, tv, p, box, stream);
    default: return launch_dv<256, false>(tq, tk, tv, p, box, stream);
    }
}

}  // namespace dflash
