// What the two tensor-core kernels of attention over an e4m3 cache share: the stages of shared memory that K and V pass
// through, and the warps that fill them.
//
// K and V come as they are, by TMA, into rings of 16 KB stages, 128 keys x 128 dims of e4m3 in 128-byte rows with the
// 128-byte swizzle. K's stages are operands of kind::f8f6f4 MMAs as they stand, and so are V's in the kernel for few rows.
// In the one for many they are widened to fp16 (exact) by four warps into a ring of its own, stages of 64 keys x 128 dims as
// two slabs of 64 dims (or 128 keys x 64 dims, one slab).
//
// Q. bf16 has 8 significant bits and e4m3 has 4, so a row of q, scaled by a power of two that brings its largest
// magnitude into (224, 448], is the sum of two e4m3 numbers: exact down to 2^-10 of the largest, off by at most 2^-10 on
// that scale below, 2^-17.8 of the largest (e4m3's steps end at 2^-9). K then needs no conversion, which would cost three times its bytes of
// shared memory traffic, and the two products run at twice the rate of one in 16 bits. A page's key scale multiplies
// its scores in fp32.
//
// V. P in e4m3 would lose small probabilities beside a large one (a first token of no value that takes half of the weight:
// what counts is then some 2^-18 of it each), hence fp16, or three e5m2 numbers. The value scale of a page goes into the exponent,
//   P' = 2^(x + log2 vs - m'), m' the lazy maximum of x + log2 vs,
// so that P' is rounded relative to the largest p vs of its row, whatever the scales are; the row sum adds P' / vs in fp32.
//
// P' is 0 below 2^-126, and then so is P' / vs, where its key's weight need not be small. So that holds for scales within
// [2^-40, 2^24] times a reference, 1 or what the CTA's first tile has, among which no weight above 2^-62 of its row's largest is
// lost; vs is relative to the reference, and the output is multiplied by it. Scales up to 2^-126, those of pages of zeros, count as
// 2^-40 of it. A piece with any other scale is worked out once more on the CUDA cores when the CTA is done with all of its
// pieces, from q, K and V as they are (far_pieces): the loops above know nothing of it. (A second sum of weights in them, which some
// five forms of cost chunks of 256 queries 3 to 14 % and blocks with a window 2 to 11 % without ever being formed: their code is
// fetched every time, and their registers are all in use. This way it is 2 % of the latter, 0.6 us, and nothing elsewhere.)
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "cache8.h"
#include "e4m3.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace dflash {
namespace tc8 {

using namespace ptx;

constexpr int kTile = 128;
constexpr int kGroup = 8;  // keys that are sure to lie in one page
constexpr int kGroups = kTile / kGroup;
constexpr int kStageBytes = 16384;
constexpr int kMaxStages = 8;  // of each ring
constexpr int kScaleRing = 8;  // tiles
constexpr float kNearLow = -40.f, kNearHigh = 24.f;  // logarithms of the value scales that P' and the row sums take (Near)
constexpr float kZeros = 0x1p-126f;                  // value scales up to this are those of pages of zeros
constexpr int kConverters = 4;
// warps behind the 8 of the softmax
constexpr int kKWarp = 8;
constexpr int kVWarp = 9;
constexpr int kMmaWarp = 10;
constexpr int kScaleWarp = 11;
constexpr int kConvertWarp = 12;
constexpr int kThreads = 32 * (kConvertWarp + kConverters);
// Registers: 16 warps at launch have 128 each, four warpgroups of them 512 a lane; the softmax takes what the others give.
constexpr int kSoftmaxRegs = 160, kOtherRegs = 96;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs <= 4 * 128, "more would wait forever");
constexpr int kSmemMax = 227 * 1024;
constexpr unsigned long long kDrainNs = 100000000ull;  // bound of the waits for work in flight after a failed one
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Shape {
    int32_t k_stages, r_stages, v_stages;  // depths of the rings: K, V as it comes, V in fp16
    int32_t q_rows;                        // rows of Q in shared memory, a multiple of 8
    int32_t box;                           // tokens per TMA box
    uint32_t page_magic;                   // page of 8-key group i: umulhi(i, page_magic), or i itself where 0
};

// A piece of the range (tree_attn.cuh) as the warp roles need it.
struct Piece {
    int32_t b, g;              // request and KV head
    int32_t n, ctx, L, lo;     // queries, keys before them, keys, first key that a query sees
    int32_t first_key, tiles;  // first key of the piece's tiles, and how many there are
    int32_t whole, slot;       // whether it is a whole pair; else its partial's slot
};
// The walk over them is one warp's, which leaves a table in shared memory: inlined into every role it made the kernels 120 to
// 200 KB of code, and the warps waited for instructions.
constexpr int kPieces = 32;

struct Pipe {
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];
    uint64_t r_full[kMaxStages], r_empty[kMaxStages];
    uint64_t v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t sc_full[kScaleRing], sc_free[kScaleRing];
    uint64_t q_full, q_free;
    uint64_t s_full[2], p_half[2], p_full[2], p_free[2];
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
    alignas(16) float k_scale[kScaleRing][kGroups];  // of a tile's groups of keys (read four at a time)
    alignas(16) float v_log[kScaleRing][kGroups];    // log2 of the value scale
    alignas(16) float v_inv[kScaleRing][kGroups];    // 2^-v_log
    float q_scale[2][128];                           // of a row of Q, by the piece's parity; NaN: the row is not finite
    int32_t par[DFLASH_MAX_TREE_NODES];
    int32_t pieces, more;
    Piece piece[kPieces];
    int32_t far;  // a piece had a value scale too far from the CTA's reference
    float v_ref;  // that, a power of two
};

// Bounded wait, of little code: false when it ran out (recorded) or another warp has given up. The test suspends the warp, so
// that the issue slots and the shared memory pipe are the working warps'.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                         unsigned long long limit)
{
    unsigned long long t0 = 0;
#pragma unroll 1
    for (uint32_t k = 0; !mbar_try_wait(bar, parity); ++k) {
        if ((k & 7u) != 0) continue;
        const unsigned long long now = globaltimer();
        if (k == 0) t0 = now;
        if (*abort_flag) return false;
        if (now - t0 > limit) {
            *abort_flag = 1;
            raise_error(err, DFLASH_DEVERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// Several barriers looked at together: their tests overlap, where waits one by one cost some 100 cycles each even when
// everything is ready. A warp's answer; what has not completed is waited for.
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity) { return mbar_test_wait(bar, parity); }

// D (TMEM) (+)= A (shared memory) . B (shared memory), e4m3
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum)
        : "memory");
}

// Instruction descriptors of fp32 accumulation: over 8-bit operands (A e4m3, B e4m3 or e5m2), and over fp16 ones, whose type
// fields are 0 too.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_mn, int b_mn, int b_e5m2)
{
    return (1u << 4) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) { return idesc_f8(M, N, a_mn, b_mn, 0); }

__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
}
__device__ __forceinline__ void give_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

// One thread sets the barriers up; what differs is how many arrivals complete a phase.
__device__ __forceinline__ void init_pipe(Pipe& ms, int r_empty_count, int p_half_count, int p_full_count)
{
    for (int i = 0; i < kMaxStages; ++i) {
        mbar_init(ms.k_full + i, 1);
        mbar_init(ms.k_empty + i, 1);
        mbar_init(ms.r_full + i, 1);
        mbar_init(ms.r_empty + i, r_empty_count);
        mbar_init(ms.v_full + i, kConverters);
        mbar_init(ms.v_empty + i, 1);
    }
    for (int i = 0; i < kScaleRing; ++i) {
        mbar_init(ms.sc_full + i, 1);
        mbar_init(ms.sc_free + i, 8);  // a softmax warp each
    }
    mbar_init(&ms.q_full, kConverters);
    mbar_init(&ms.q_free, 1 + 8);  // the MMAs of the piece's last scores, and a softmax warp each that has read the rows' scales
    for (int i = 0; i < 2; ++i) {
        mbar_init(ms.s_full + i, 1);
        mbar_init(ms.p_half + i, p_half_count);
        mbar_init(ms.p_full + i, p_full_count);
        mbar_init(ms.p_free + i, 1);
    }
    mbar_init(&ms.drain, 1);
    ms.abort = 0;
    ms.far = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// 8 columns of 32 values, one a lane -> in lanes l, l + 8, ... the maximum (sum) of column l.
template <bool kSum>
__device__ __forceinline__ float transpose8(float (&v)[8], int lane)
{
    auto join = [](float a, float b) { return kSum ? a + b : fmaxf(a, b); };
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float send = upper ? v[i] : v[i + off];
            const float keep = upper ? v[i + off] : v[i];
            v[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
    }
    v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 8));
    return join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// Fills the table with the walk's next pieces (a whole warp; the others wait).
__device__ __forceinline__ void list_pieces(const TreeAttnParams& p, PieceWalk& w, Pipe& ms)
{
    int32_t n = 0;
#pragma unroll 1
    for (; n < kPieces && !w.done(); w.next(p), ++n) {
        if ((threadIdx.x & 31) == 0)
            ms.piece[n] = Piece{w.b, w.g, w.req.n, w.req.ctx, w.req.L, w.req.lo, (w.req.tile0 + w.t0) * kTile, w.t1 - w.t0,
                                w.whole(), w.slot()};
    }
    if ((threadIdx.x & 31) == 0) {
        ms.pieces = n;
        ms.more = !w.done();
    }
}

// Runs a warp role over the range's pieces that have queries of this tile. Every role goes through the same tables, and
// the whole CTA meets between them: a role that has given up goes on without work.
template <typename Body>
__device__ __forceinline__ void each_piece(const TreeAttnParams& p, PieceWalk& w, int32_t node0, Pipe& ms, bool lists, Body body)
{
#pragma unroll 1
    for (;;) {
        const int32_t n = ms.pieces;
        const bool more = ms.more != 0;
#pragma unroll 1
        for (int32_t i = 0; i < n; ++i) {
            const Piece pc = ms.piece[i];
            if (pc.n > node0) body(pc);
        }
        if (!more) return;
        asm volatile("barrier.sync 0;" ::: "memory");
        if (lists) list_pieces(p, w, ms);
        asm volatile("barrier.sync 0;" ::: "memory");
    }
}

// Page id of a key (a multiple of 8) as the table has it, and its slot.
__device__ __forceinline__ int32_t page_id(const TreeAttnParams& p, const Shape& x, int32_t b, int32_t key, int32_t& slot)
{
    const uint32_t group = (uint32_t)key / kGroup;
    const int32_t pg = (int32_t)(x.page_magic ? __umulhi(group, x.page_magic) : group);
    slot = key - pg * p.page_size;
    return __ldg(p.page_table + (int64_t)b * p.max_pages + pg);
}

// The value scales that P' takes beside a reference: those of pages of zeros, and [low, high].
struct Near {
    float zeros, low, high;
    __device__ __forceinline__ explicit Near(float ref)
        : zeros(ref > 1.f ? -0.5f : kZeros), low(ref * exp2f(kNearLow)), high(ref * exp2f(kNearHigh))
    {
        // (beside a reference above 1 a page of zeros would no longer be next to nothing)
    }
    __device__ __forceinline__ bool lacks(float scale) const { return scale > zeros && !(scale >= low && scale <= high); }
};

// A producer warp: K or V by TMA. Boxes without a visible key are fetched at an out-of-bounds page, which the TMA unit fills
// with zeros. Page ids are asked for a tile ahead. `wait`: a warp's bounded wait.
template <typename Wait>
__device__ __forceinline__ void produce(const TreeAttnParams& p, const Shape& x, PieceWalk& w, int32_t node0, Pipe& ms,
                                        const CUtensorMap* map, uint8_t* ring, uint64_t* full, uint64_t* empty, int32_t depth,
                                        Wait wait)
{
    const int lane = threadIdx.x & 31;
    const uint64_t policy = l2_policy_evict_first();
    const int32_t boxes = kTile / x.box, chunks = (p.D + 127) / 128;
    RingPos pos{0, 0u};
    uint32_t issued = 0, phase = 0;
    bool ok = true;
    each_piece(p, w, node0, ms, false, [&](const Piece& pc) {
        const int32_t n = pc.tiles;
        // this lane's box of tile t: whether it holds a visible key, its page as the table has it and its slot there
        auto box_of = [&](int32_t t, int32_t& slot, bool& live) -> int32_t {
            const int32_t key = pc.first_key + t * kTile + lane * x.box;
            slot = 0;
            live = false;
            if (lane >= boxes || t >= n || key >= pc.L || key + x.box <= pc.lo) return p.num_pages;
            live = true;
            return page_id(p, x, pc.b, key, slot);
        };
        int32_t next_slot;
        bool next_live;
        int32_t next = box_of(0, next_slot, next_live);
#pragma unroll 1
        for (int32_t t = 0; t < n && ok; ++t) {
            const int32_t slot = next_slot;
            const bool live = next_live;
            int32_t page = next;
            next = box_of(t + 1, next_slot, next_live);
            if (live && (page < 0 || page >= p.num_pages)) {
                raise_error(p.err, DFLASH_DEVERR_PAGE_ID);
                page = p.num_pages;
            }
#pragma unroll 1
            for (int32_t c = 0; c < chunks; ++c) {
                ok = wait(empty + pos.idx, pos.phase ^ 1u);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(full + pos.idx, kStageBytes);
                __syncwarp();
                if (lane < boxes) {
                    uint8_t* dst = ring + (size_t)pos.idx * kStageBytes + lane * x.box * 128;
                    // read once: the first to leave L2, unless other query tiles read it again
                    if (p.n_sub == 1)
                        tma_load_4d_hint(dst, map, full + pos.idx, c * 128, pc.g, slot, page, policy);
                    else
                        tma_load_4d(dst, map, full + pos.idx, c * 128, pc.g, slot, page);
                }
                __syncwarp();
                issued |= 1u << pos.idx;
                phase = (phase & ~(1u << pos.idx)) | (pos.phase << pos.idx);
                pos.advance(1, depth);
            }
        }
    });
    // no copy of ours may land after the CTA has gone, whichever wait of it has run out
    if (lane == 0) {
        const unsigned long long t0 = globaltimer();
        for (int s = 0; s < depth; ++s)
            if (issued & (1u << s))
                while (!mbar_test_wait(full + s, (phase >> s) & 1u) && globaltimer() - t0 < kDrainNs) {
                }
    }
    __syncwarp();
}

// What a CTA's value scales are relative to: 1 where its first tile's largest one is ordinary, else the power of two below that (a
// whole warp, a scale a lane). Its logarithm.
__device__ __forceinline__ int32_t reference(float v_scale)
{
    const int32_t none = -1000, top = __reduce_max_sync(0xffffffffu, v_scale > kZeros ? __float2int_rd(log2f(v_scale)) : none);
    return top == none || (top >= -24 && top <= 16) ? 0 : min(max(top, -70), 100);
}

// The scale warp: the scales of a tile's groups of keys, a lane each; ids two tiles ahead and scales one.
template <typename Wait>
__device__ __forceinline__ void fetch_scales(const TreeAttnParams& p, const Shape& x, PieceWalk& w, int32_t node0, Pipe& ms,
                                             Wait wait)
{
    const int lane = threadIdx.x & 31;
    RingPos pos{0, 0u};
    bool ok = true, first = true;
    float ref = 0.f;
    Near near(1.f);
    each_piece(p, w, node0, ms, true, [&](const Piece& pc) {
        const int32_t n = pc.tiles;
        auto group_page = [&](int32_t t) -> int32_t {
            const int32_t key = pc.first_key + t * kTile + lane * kGroup;
            if (lane >= kGroups || t >= n || key >= pc.L || key + kGroup <= pc.lo) return -1;
            int32_t slot;
            return page_id(p, x, pc.b, key, slot);
        };
        auto scales_of = [&](int32_t page, float& ks, float& vs) {
            ks = 1.f, vs = -1.f;  // keys that nobody sees, or zeros
            if (page < 0 || page >= p.num_pages) return;
            const int64_t at = (int64_t)page * p.Hkv + pc.g;
            ks = __ldg(p.k_scale + at);
            vs = __ldg(p.v_scale + at);
        };
        float ks, vs;
        scales_of(group_page(0), ks, vs);
        int32_t next_page = group_page(1);
        if (first) {
            first = false;
            const int32_t e = reference(vs);
            ref = (float)e;
            near = Near(power_of_two(e));
            if (lane == 0) ms.v_ref = power_of_two(e);
        }
#pragma unroll 1
        for (int32_t t = 0; t < n && ok; ++t) {
            float next_ks, next_vs;
            scales_of(next_page, next_ks, next_vs);
            next_page = group_page(t + 2);
            if (near.lacks(vs)) ms.far = 1;
            const float v_log = fminf(fmaxf(log2f(vs) - ref, kNearLow), kNearHigh);  // (kNearLow for vs < 0)
            ok = wait(ms.sc_free + pos.idx, pos.phase ^ 1u);
            if (!ok) break;
            if (lane < kGroups) {
                ms.k_scale[pos.idx][lane] = ks;
                ms.v_log[pos.idx][lane] = v_log;
                ms.v_inv[pos.idx][lane] = exp2f(-v_log);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ms.sc_full + pos.idx);
            pos.advance(1, kScaleRing);
            ks = next_ks;
            vs = next_vs;
        }
    });
}

// A piece's rows of Q, split into two e4m3 numbers each by the four warps of `ct` (0 .. 127). Q lies as
// [128-dim chunk][hi, lo][q_rows][128 bytes], 128-byte swizzle. A row is a warp's, in one or two loads, or half a warp's up to
// 128 dims. Little code, as it runs once a piece and is fetched each time: a warp per row of 128 dims with two rows in flight took
// 44000 cycles for 128 rows before the first score of a piece (256 queries of 2 requests: 202 us in place of 152), 8 and 16
// rows of half a warp in flight 159 and 168 us.
template <bool kHalf, int kLoads>
__device__ __forceinline__ void split_queries(const TreeAttnParams& p, const Shape& x, const Piece& pc, const SubTile& st,
                                              int32_t node0, Pipe& ms, uint8_t* q_s, int ct, uint32_t parity)
{
    constexpr int kLanes = kHalf ? 16 : 32;
    const int lane = ct & (kLanes - 1);
    const int32_t kc_n = (p.D + 127) / 128;
    const uint32_t q_chunk_bytes = (uint32_t)x.q_rows * 128;
    const int32_t live = min(p.npt, pc.n - node0) * p.Gc;
#pragma unroll 1
    for (int32_t row0 = 0; row0 < live; row0 += 128 / kLanes) {
        const int32_t row = row0 + ct / kLanes, nd = row / p.Gc;
        if (__all_sync(0xffffffffu, row >= live)) break;
        const __nv_bfloat16* src =
            static_cast<const __nv_bfloat16*>(p.q) +
            (((int64_t)pc.b * p.T + node0 + nd) * p.Hq + pc.g * p.G + st.gc * p.Gc + (row - nd * p.Gc)) * p.D;
        uint4 v[kLoads];
        float amax = 0.f;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int32_t d = (k * kLanes + lane) * 8;
            v[k] = row < live && d < p.D ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const uint32_t q[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float a = fabsf(u2f(q[u] << 16)), b = fabsf(u2f(q[u] & 0xFFFF0000u));
                amax = fmaxf(amax, fmaxf(a, b));
                bad |= !(a < INFINITY) || !(b < INFINITY);
            }
        }
        if (bad) amax = INFINITY;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const int32_t e = e4m3_exponent(amax);
        const float inv = power_of_two(-e);
        if (row < live) {
            if (lane == 0) ms.q_scale[parity][row] = amax == INFINITY ? NAN : power_of_two(e);
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int32_t d = (k * kLanes + lane) * 8;
                if (d >= kc_n * 128) continue;
                const uint32_t q[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float f[4], g[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[2 * i] = u2f(q[2 * u + i] << 16) * inv;
                        f[2 * i + 1] = u2f(q[2 * u + i] & 0xFFFF0000u) * inv;
                    }
                    hi[u] = e4m3x4(f[0], f[1], f[2], f[3]);
                    e4m3_values(hi[u], g);
                    lo[u] = e4m3x4(f[0] - g[0], f[1] - g[1], f[2] - g[2], f[3] - g[3]);
                }
                uint8_t* dst = q_s + (d >> 7) * 2 * q_chunk_bytes + row * 128 + ((((d & 127) >> 4) ^ (row & 7)) << 4) + (d & 8);
                *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(dst + q_chunk_bytes) = make_uint2(lo[0], lo[1]);
            }
        }
        __syncwarp();
    }
    fence_proxy_async_smem();
    __syncwarp();
    if ((ct & 31) == 0) mbar_arrive(&ms.q_full);
}

// The four warps that do no more than that.
template <typename Wait>
__device__ __forceinline__ void split_all(const TreeAttnParams& p, const Shape& x, PieceWalk& w, const SubTile& st,
                                          int32_t node0, Pipe& ms, uint8_t* q_s, Wait wait)
{
    uint32_t q_phase = 0;
    bool ok = true;
    each_piece(p, w, node0, ms, false, [&](const Piece& pc) {
        if (ok) ok = wait(&ms.q_free, q_phase ^ 1u);  // the last piece's scores are computed, long before it is done
        if (!ok) return;
        split_queries<false, 2>(p, x, pc, st, node0, ms, q_s, threadIdx.x - kConvertWarp * 32, q_phase);
        q_phase ^= 1u;
    });
}

// The four warps that also widen V: a piece's Q once the last piece's scores are computed, then V's stages. kVN: dims of a
// widened stage (128, or 64 of one slab); kDims: the most of a head, at most 256.
template <int kVN, int kDims, typename Wait>
__device__ __forceinline__ void convert(const TreeAttnParams& p, const Shape& x, PieceWalk& w, const SubTile& st, int32_t node0,
                                        Pipe& ms, uint8_t* q_s, const uint8_t* r_ring, uint8_t* v_ring, Wait wait)
{
    constexpr int kVKeys = kVN == 64 ? 128 : 64;       // keys of a widened stage
    constexpr int kChunks = kVN / 16;                  // 16-byte pieces of its rows as they come
    constexpr int kRows = 32 * kConverters / kChunks;  // rows that the warps take at once
    static_assert(kVKeys / kRows == 4, "four rows of a stage per thread");
    const int ct = threadIdx.x - kConvertWarp * 32, lane = ct & 31;
    const int vc = ct % kChunks, vr = ct / kChunks;
    RingPos rp{0, 0u}, vp{0, 0u};
    uint32_t q_phase = 0;
    bool ok = true;
    each_piece(p, w, node0, ms, false, [&](const Piece& pc) {
        if (ok) ok = wait(&ms.q_free, q_phase ^ 1u);
        if (!ok) return;
        split_queries<(kDims <= 128), 1>(p, x, pc, st, node0, ms, q_s, ct, q_phase);
        q_phase ^= 1u;
        const int32_t n = pc.tiles, chunks = (p.D + 127) / 128;
#pragma unroll 1
        for (int32_t t = 0; t < n && ok; ++t) {
            const int32_t key0 = pc.first_key + t * kTile;
            // rows of V that no query sees are zeroed: 0 x NaN would reach every row
            const bool edge = key0 < pc.lo || key0 + kTile > pc.L;
#pragma unroll 1
            for (int32_t c = 0; c < chunks && ok; ++c) {
                ok = wait(ms.r_full + rp.idx, rp.phase);
                if (!ok) break;
                const uint8_t* src = r_ring + (size_t)rp.idx * kStageBytes;
                constexpr int kHalves = kTile / kVKeys;
                uint4 in[kHalves][4];
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = h * kVKeys + vr + k * kRows;
                        in[h][k] = *reinterpret_cast<const uint4*>(src + row * 128 + ((vc ^ (row & 7)) << 4));
                        if (edge && (key0 + row < pc.lo || key0 + row >= pc.L)) in[h][k] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    if (ok) ok = wait(ms.v_empty + vp.idx, vp.phase ^ 1u);
                    if (!ok) break;
                    uint8_t* stage = v_ring + (size_t)vp.idx * kStageBytes;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = vr + k * kRows;
                        const uint32_t q[4] = {in[h][k].x, in[h][k].y, in[h][k].z, in[h][k].w};
                        uint32_t f[8];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            f[2 * u] = e4m3_to_f16(q[u]);
                            f[2 * u + 1] = e4m3_to_f16(q[u] >> 16);
                        }
                        // the second slab's lanes write their halves the other way round, so that eight lanes meet
                        // eight banks
                        const int slab = vc >> 2, c2 = (vc & 3) * 2;
                        uint8_t* dst = stage + slab * (kVKeys * 128) + row * 128;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int ii = i ^ slab;
                            *reinterpret_cast<uint4*>(dst + (((c2 + ii) ^ (row & 7)) << 4)) =
                                ii ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(ms.v_full + vp.idx);
                        if (h == kHalves - 1) mbar_arrive(ms.r_empty + rp.idx);
                    }
                    vp.advance(1, x.v_stages);
                }
                rp.advance(1, x.r_stages);
            }
        }
    });
}

// Rows [row0, row0 + R) of a piece on the CUDA cores in fp32, 8 keys a step: a warp's lanes share the dims (kWords words of four), and the
// keys of a step once the dots are added up. m is a row's running maximum, l a lane's part of its sum.
template <int kWords, int R>
__device__ __forceinline__ void far_rows(const TreeAttnParams& p, const Shape& x, const TreeReq& req, int32_t b, int32_t g, int32_t first,
                                         int32_t end, bool whole, int32_t head0, int32_t node0, int32_t row0, int32_t live,
                                         int64_t prow, const int32_t* lo_s, const uint32_t* anc_s)
{
    const int lane = threadIdx.x & 31, words = (p.T + 31) / 32;
    const float scale = p.scale * kLog2e;
    auto out_row = [&](int32_t row) -> int64_t {
        const int32_t nd = row / p.Gc;
        return ((int64_t)b * p.T + node0 + nd) * p.Hq + head0 + (row - nd * p.Gc);
    };
    float q[R][kWords][4], acc[R][kWords][4], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t orow = out_row(min(row0 + r, live - 1));  // (rows behind the last repeat it and are not written)
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
            const int32_t d = c * 128 + lane * 4;
            const uint2 v = d < p.D ? __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + orow * p.D + d))
                                    : make_uint2(0, 0);
            q[r][c][0] = u2f(v.x << 16), q[r][c][1] = u2f(v.x & 0xFFFF0000u);
            q[r][c][2] = u2f(v.y << 16), q[r][c][3] = u2f(v.y & 0xFFFF0000u);
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[r][c][u] = 0.f;
        }
    }
#pragma unroll 1
    for (int32_t key0 = first; key0 < end; key0 += kGroup) {
        if (key0 + kGroup <= req.lo) continue;
        int32_t slot;
        const int32_t page = page_id(p, x, b, key0, slot);
        const bool good = page >= 0 && page < p.num_pages;  // (else its keys read as zeros, and the error is raised)
        const int64_t scale_at = (int64_t)page * p.Hkv + g;
        const float ks = good ? __ldg(p.k_scale + scale_at) : 0.f, vs = good ? __ldg(p.v_scale + scale_at) : 0.f;
        const int64_t at = (int64_t)page * p.sp + (int64_t)slot * p.ss + (int64_t)g * p.sh;
        auto load = [&](const void* base, uint32_t (&w)[kGroup][kWords]) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
#pragma unroll
                for (int c = 0; c < kWords; ++c) {
                    const int32_t d = c * 128 + lane * 4, key = key0 + k;
                    w[k][c] = 0u;  // (keys that nobody sees may hold anything)
                    if (good && key >= req.lo && key < end && d < p.D)
                        w[k][c] = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + at + k * p.ss + d));
                }
        };
        uint32_t kw[kGroup][kWords], vw[kGroup][kWords];
        load(p.k, kw);
        if (kWords < 4) load(p.v, vw);  // (on its way; registers for a wide head's do not reach)
        float dot[R][8];
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            float f[kWords][4];
#pragma unroll
            for (int c = 0; c < kWords; ++c) e4m3_values(kw[k][c], f[c]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                dot[r][k] = 0.f;
#pragma unroll
                for (int c = 0; c < kWords; ++c)
#pragma unroll
                    for (int u = 0; u < 4; ++u) dot[r][k] = fmaf(q[r][c][u], f[c][u] * ks, dot[r][k]);
            }
        }
        if (kWords == 4) load(p.v, vw);
        float weight[R];  // of key `lane & 7`, times its value scale
        const int32_t key = key0 + (lane & 7), a = key - req.ctx;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int32_t nd = min(row0 + r, live - 1) / p.Gc;
            const bool on = key < end && (a < 0 ? key >= lo_s[nd] : ((anc_s[nd * words + (a >> 5)] >> (a & 31)) & 1u) != 0);
            float y = transpose8<true>(dot[r], lane) * scale;
            y = on ? y : -INFINITY;
            float top = y;
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            if (top > m[r]) {  // (the same for the whole warp)
                const float alpha = ex2(m[r] - top);  // 0 from -inf
                m[r] = top;
                l[r] *= alpha;
#pragma unroll
                for (int c = 0; c < kWords; ++c)
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[r][c][u] *= alpha;
            }
            const float e = on ? ex2(y - m[r]) : 0.f;
            l[r] += e;
            weight[r] = e * vs;
        }
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            float f[kWords][4];
#pragma unroll
            for (int c = 0; c < kWords; ++c) e4m3_values(vw[k][c], f[c]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float e = __shfl_sync(0xffffffffu, weight[r], k);
#pragma unroll
                for (int c = 0; c < kWords; ++c)
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[r][c][u] = fmaf(e, f[c][u], acc[r][c][u]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int32_t row = row0 + r;
        float sum = l[r];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (row >= live) continue;
        const int64_t orow = out_row(row);
        const float inv = tree_inv_sum(sum, whole), lse = tree_row_lse((m[r] + log2f(sum)) * kLn2, sum, whole);
        if (lane == 0 && !whole) p.part_lse[prow + row] = lse;
        if (lane == 0 && whole && p.lse) p.lse[orow] = lse;
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
            const int32_t d = c * 128 + lane * 4;
            if (d >= p.D) continue;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (!whole)
                    p.part_out[(prow + row) * p.DV + d + u] = acc[r][c][u] * inv;
                else
                    static_cast<__nv_bfloat16*>(p.out)[orow * p.D + d + u] = __float2bfloat16_rn(acc[r][c][u] * inv);
            }
        }
    }
}

// The pieces of a range with a value scale that P' does not take, in place of what the tensor cores have left there. Called by the 8
// warps of the softmax when every role is done; each walks the range by itself. A warp takes as many rows at once as its registers
// hold: 256 queries of 2 requests of 8192 keys, 32/8 heads of 128, take 7 ms, 75 ms a row at a time. (As a function that is called it
// took registers of the loops before it: single tokens on long contexts 193 us in place of 183.)
__device__ __forceinline__ void far_pieces(const TreeAttnParams& p, uint32_t page_magic, int32_t range, int32_t sub,
                                               float ref, int32_t* par_s, int32_t* lo_s, uint32_t* anc_s)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SubTile st = sub_tile(p, sub);
    const int32_t node0 = st.rt * p.npt;
    const Near near(ref);
    Shape x{};
    x.page_magic = page_magic;
    PieceWalk w;
    w.start(p, range);
#pragma unroll 1
    for (; !w.done(); w.next(p)) {
        const TreeReq req = w.req;
        if (req.n <= node0) continue;
        const int32_t first = (req.tile0 + w.t0) * kTile, end = min(req.L, (req.tile0 + w.t1) * kTile);
        // the pages that some query sees, as the scale warp takes them
        bool far = false;
#pragma unroll 1
        for (int32_t key = first + lane * kGroup; key < end; key += 32 * kGroup) {
            if (key + kGroup <= req.lo) continue;
            int32_t slot;
            const int32_t page = page_id(p, x, w.b, key, slot);
            if (page >= 0 && page < p.num_pages) far |= near.lacks(__ldg(p.v_scale + (int64_t)page * p.Hkv + w.g));
        }
        if (!__any_sync(0xffffffffu, far)) continue;  // (the same for all warps)
        named_bar_sync_256();
        tree_load_parents(p, w.b, req.n, par_s, tid, 256);
        named_bar_sync_256();
        tree_walk_nodes(p, req, node0, min(p.npt, req.n - node0), par_s, anc_s, lo_s, tid, 256);
        named_bar_sync_256();
        const int32_t live = min(p.npt, req.n - node0) * p.Gc, head0 = w.g * p.G + st.gc * p.Gc;
        const bool whole = w.whole();
        const int64_t prow = tree_part_row(p, range, sub, w.slot());
        auto rows = [&](auto words, auto at_once) {
            constexpr int R = decltype(at_once)::value;
#pragma unroll 1
            for (int32_t row = warp * R; row < live; row += 8 * R)
                far_rows<decltype(words)::value, R>(p, x, req, w.b, w.g, first, end, whole, head0, node0, row, live, prow, lo_s,
                                                    anc_s);
        };
        if (p.D <= 128)
            rows(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
        else if (p.D <= 256)
            rows(std::integral_constant<int, 2>(), std::integral_constant<int, 2>());
        else
            rows(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    }
}

// ------------------------------------------------------------------------------- host side

// The kernel for few query rows (cache8_attn_few.cu).
cudaError_t launch_few(const CUtensorMap& tk, const CUtensorMap& tv, const TreeAttnParams& p, Shape x, cudaStream_t stream);

// Tensor maps of K and V: boxes of 128 dims of `box` tokens of one page. False: the driver has no such map.
bool encode_maps(const TreeAttnParams& p, int32_t box, CUtensorMap* tk, CUtensorMap* tv);

// The ring depths for what Q, P and the rest leave of shared memory. False: too little for the smallest.
inline bool deal_stages(Shape& x, int32_t bytes_left)
{
    const int32_t stages = bytes_left / kStageBytes;
    if (stages < 4) return false;
    x.v_stages = std::min(4, std::max(1, stages / 3));
    x.r_stages = std::min(kMaxStages, (stages - x.v_stages) / 2);
    x.k_stages = std::min(kMaxStages, stages - x.v_stages - x.r_stages);
    return true;
}

}  // namespace tc8
}  // namespace dflash
