// Log probabilities of given tokens, entropy and the top tokens of rows of logits, in one pass.
//
//   m = max_v l_v, y_v = (l_v - m) log2(e) / temperature, s = sum_v 2^y_v, w = sum_v y_v 2^y_v
//   log_z = m / temperature + ln s,  logp(v) = (l_v - m) / temperature - ln s,  entropy = ln s - ln 2 * w / s
// Sums are taken about the running maximum, which is subtracted from the logit itself before the scaling: the
// differences stay exact to fp32 whatever the size of the logits. In a row with one likely token s is 1, the
// maximum's own term, and the mass p of all the others: each of these is added to it once, off by at most what is
// added (and by 2^-24), so that ln s loses p at most, where p is below 2^-24 all of it. The top token's logp is 0 then,
// and the entropy p (1 - ln p) is p low, a twentieth of it: w, without a term of the maximum's, is exact to fp32.
//
// A row is cut into equal slices, a CTA of 128 threads each, streamed in steps of 16 values a thread with the
// next step's loads in flight; no barrier until its end. Beside the sums a thread keeps the maximum of each
// thirty-second of its steps: of a group of values.
//
// Selection. A value and its id form a 64-bit key (order-preserving image of the value above the id's
// complement), all distinct, so "the k largest keys" is the definition. At the slice's end the threads' maxima
// give a bound that k values or more reach. Only groups whose maximum reaches it are read again (some 70 to 100
// of 4096 for k = 64), and only their values that reach it become candidates. Candidates and kept keys are
// ranked against each other (a key's rank is the number of larger ones; no sort) and the first k stay. The
// buffer holds 256 candidates of each warp; a warp that might add more waits for a merge, so nothing but the
// time depends on the data: a row of equal logits reads every group again. A thread's values of a step are
// whole sectors, so that reading a group again fetches little beside it.
//
// Measured in replayed graphs on inputs beyond L2, k = 64 beside none: 1000 rows of 151937 fp32 117 and 95 us
// (floor 90), of 151936 bf16 76 and 61 (45); 4000 rows of 32000 bf16 93 and 57 (38); 8 rows of 151936 bf16 18 and
// 6; 1 row fp32 16. Bound: fp32 the stream, then the groups read again, with no loads of the row ahead meanwhile;
// bf16 the issue slots: a value costs what it costs in fp32, whose kernel issues in 54 us of its time for the first
// of these sizes, which 45 us of stream do not hide. Rows a little above whole waves of CTAs (eight an SM) leave
// the last wave mostly idle: 1216 rows of 151936 bf16 without top tokens 67 us, 1230 rows 101.
//
// (Earlier forms, timed call by call after a flush of L2, where this one took 117 us for the first size: candidates
// picked step by step, with a sort of 256 per merge, 460; merges by rank at every doubling of what has been seen
// 143; 16 groups a thread in place of 32 137. A bound from all four warps alone, and a short last slice, took 43 us for
// the 8 rows in place of 27: a warp without values left no bound.)
//
// Slices leave their sums and keys in the workspace; the last CTA of a row to arrive (a counter, no waiting)
// merges them the same way and writes the row.
#include <algorithm>
#include <cmath>

#include "dflash_device.cuh"
#include "tree.h"

namespace dflash {
namespace {

constexpr int kThreads = 128;
constexpr int kElems = 16;      // values per thread and step
constexpr int kCtasPerSm = 8;
constexpr int kSliceElems = kElems * kThreads;  // a step
constexpr int kMaxK = DFLASH_MAX_TOP_K;
constexpr int kWarpRoom = 256;  // candidates a warp may add between merges: 32 vectors of bf16 at least
constexpr int kCand = kThreads / 32 * kWarpRoom + 512;  // what may wait, and what may come before it is looked at
constexpr int kAgain = 4;  // vectors read again at once, per thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned long long Key;

__device__ __forceinline__ Key make_key(float x, uint32_t id)
{
    uint32_t u = __float_as_uint(x + 0.f);  // -0 -> +0
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((Key)u << 32) | (0xFFFFFFFFu - id);
}

__device__ __forceinline__ float key_value(Key k)
{
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

__device__ __forceinline__ int32_t key_id(Key k) { return (int32_t)(0xFFFFFFFFu - (uint32_t)k); }

// 2^x on the special-function unit: 2 ulp, below the rounding of the sums
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

constexpr int kPhases = 32;  // groups per thread, a bit each
constexpr int kList = kPhases / 2 * kThreads;

// (17 KB a CTA: with 25 KB, eight to an SM, the loads in flight had too little of the L1 left: 104 -> 133 us without
// top tokens.)
struct Shared {
    Key kept[kMaxK];  // the k largest so far, largest first
    union {
        __nv_bfloat16 group[kPhases][kThreads];  // maxima rounded up, until it is known which groups to read again
        Key cand[kCand];                         // then the waiting candidates
    };
    uint16_t list[kList];  // groups to read again: phase * kThreads + thread
    int32_t warp_n[kThreads / 32];
    Key bound;                // keys at or below it are out
    int32_t n_kept, n_cand;
    int32_t last;
    union {
        float warp_top[4][kThreads / 32];
        Key warp_key[4][kThreads / 32];
    };
    float red[3][kThreads / 32];
};

// Ranks the waiting candidates and the kept keys; the first k stay. Every thread of the CTA calls it after a barrier.
__device__ __forceinline__ void merge(Shared& sh, int32_t k, int tid)
{
    const int32_t n_cand = sh.n_cand;
    int32_t kept = sh.n_kept;
    const Key* cand = sh.cand;
#pragma unroll 1
    for (int32_t at = 0; at < n_cand; at += kThreads - kMaxK) {
        const int32_t here = min(n_cand - at, kThreads - kMaxK);
        Key mine = 0;
        int32_t rank = 0;
        if (tid < kept) {
            mine = sh.kept[tid];
            rank = tid;
        } else if (tid >= kMaxK && tid - kMaxK < here) {
            mine = cand[at + tid - kMaxK];
            int32_t lo = 0, hi = kept;  // kept keys are in order
            while (lo < hi) {
                const int32_t mid = (lo + hi) >> 1;
                if (sh.kept[mid] > mine)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            rank = lo;
        }
        if (mine) {
#pragma unroll 4
            for (int32_t i = 0; i < here; ++i) rank += cand[at + i] > mine;
        }
        __syncthreads();
        if (mine && rank < k) sh.kept[rank] = mine;
        kept = min(k, kept + here);
        __syncthreads();
    }
    if (tid == 0) {
        sh.n_cand = 0;
        sh.n_kept = kept;
        if (kept == k) sh.bound = max(sh.bound, sh.kept[k - 1]);
    }
    __syncthreads();
}

// A bound from one value of each thread: at least k of them reach it, or it is `none`, the least there is. For each
// number of warps j the ceil(k / j)-th largest of a warp's, and of these the j-th largest: j warps hold k values from
// there on. The best of the four is taken, so that warps without values (of a short slice) cost little.
template <typename T>
__device__ __forceinline__ T bound_of(T (&part)[4][kThreads / 32], int32_t k, int tid, T x, T none)
{
    const int lane = tid & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
        const bool down = (lane & size) == 0;
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const T other = __shfl_xor_sync(0xffffffffu, x, d);
            const bool larger = ((lane & d) == 0) == down;  // this lane takes the larger of the two
            x = larger ? (x > other ? x : other) : (x > other ? other : x);
        }
    }
#pragma unroll
    for (int j = 1; j <= 4; ++j)
        if (lane == (k + j - 1) / j - 1) part[j - 1][tid >> 5] = x;
    __syncthreads();
    T best = none;
#pragma unroll
    for (int j = 1; j <= 4; ++j) {
        if ((k + j - 1) / j > 32) continue;
        // the j-th largest of four
        const T a = part[j - 1][0], b = part[j - 1][1], c = part[j - 1][2], d = part[j - 1][3];
        const T ab = a > b ? a : b, ba = a > b ? b : a, cd = c > d ? c : d, dc = c > d ? d : c;
        const T low = ab > cd ? cd : ab, high = ba > dc ? ba : dc;  // the two between the largest and the least
        const T nth = j == 1   ? (ab > cd ? ab : cd)
                      : j == 2 ? (low > high ? low : high)
                      : j == 3 ? (low > high ? high : low)
                               : (ba > dc ? dc : ba);
        best = nth > best ? nth : best;
    }
    return best;
}

__device__ __forceinline__ void put(Shared& sh, Key key) { sh.cand[atomicAdd(&sh.n_cand, 1)] = key; }

// Element e of a 16-byte vector of E.
template <typename E>
__device__ __forceinline__ float element(const uint4& v, int e)
{
    if (sizeof(E) == 2) {
        const uint32_t x = e / 2 == 0 ? v.x : e / 2 == 1 ? v.y : e / 2 == 2 ? v.z : v.w;
        return __uint_as_float(e % 2 ? x & 0xFFFF0000u : x << 16);
    }
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
}

struct Slice {
    const void* base;         // its first sector
    int32_t nq;               // sectors (32 bytes)
    int32_t whole0, whole1;   // those that hold the row's elements only
    int32_t id0;              // id of the first element
    int32_t steps, phase_len;
};

// The k largest keys of the slice whose group maxima are in sh.group. Out of line: the stream keeps its registers.
template <typename E>
__device__ __noinline__ void select_again(Shared& sh, int32_t k, const Slice sl, float top, bool has_edge, float edge_x,
                                          int32_t edge_id)
{
    constexpr int kN = 16 / sizeof(E);
    constexpr int kVecs = kElems / kN;
    constexpr int kSecs = kVecs / 2;
    const int tid = threadIdx.x;
    // the bound: a value that k values or more reach (-inf where there are not that many)
    float limit = bound_of(sh.warp_top, k, tid, top, -INFINITY);
    uint32_t mine = 0;  // this thread's groups to read again
#pragma unroll 4
    for (int32_t phase = 0; phase * sl.phase_len < sl.steps; ++phase)
        if (__bfloat162float(sh.group[phase][tid]) >= limit) mine |= 1u << phase;
    // where a thread's groups stand in the list, and how many there are of all threads
    int32_t place = 0, n_list = 0;
    auto count = [&](uint32_t groups) {
        const int32_t n = __popc(groups);
        int32_t incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, off);
            if ((tid & 31) >= off) incl += v;
        }
        if ((tid & 31) == 31) sh.warp_n[tid >> 5] = incl;
        __syncthreads();  // (the first time also: the groups' maxima make room for candidates)
        place = incl - n;
        n_list = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < tid >> 5) place += sh.warp_n[i];
            n_list += sh.warp_n[i];
        }
    };
    count(mine);
    uint32_t rest = 0;
    const bool halves = n_list > kList;  // many equal values: half of the groups a time
    if (halves) {
        rest = mine & ~0xFFFFu;
        mine &= 0xFFFFu;
        __syncthreads();
        count(mine);
    }
    if (has_edge && edge_x >= limit) put(sh, make_key(edge_x, (uint32_t)edge_id));
    // the groups' 16-byte vectors, a group's `per` one after another, dealt to the threads four at a time
    const int32_t per = sl.phase_len * kVecs;
    Key bound = 0;
#pragma unroll 1
    for (int half = 0; half < (halves ? 2 : 1); ++half) {
        if (half) {
            mine = rest;
            count(mine);
        }
        for (; mine; mine &= mine - 1) sh.list[place++] = (uint16_t)((__ffs(mine) - 1) * kThreads + tid);
        __syncthreads();
        const int64_t total = (int64_t)n_list * per;
        int64_t from = 0;
#pragma unroll 1
        do {
            uint4 v[kAgain];
            int32_t at[kAgain];  // 16-byte vector of the slice, or -1
#pragma unroll
            for (int i = 0; i < kAgain; ++i) {
                const int64_t j = from + i * kThreads + tid;
                at[i] = -1;
                v[i] = make_uint4(0, 0, 0, 0);
                if (j < total) {
                    const int32_t e = total <= INT32_MAX ? (int32_t)j / per : (int32_t)(j / per);
                    const int32_t g = sh.list[e], vec = g / kThreads * per + (int32_t)(j - (int64_t)e * per);
                    const int32_t q = (vec >> 1) * kThreads + g % kThreads;  // its sector
                    if ((vec >> 1) < sl.steps * kSecs && q >= sl.whole0 && q < sl.whole1) {
                        at[i] = 2 * q + (vec & 1);
                        v[i] = __ldg(static_cast<const uint4*>(sl.base) + at[i]);
                    }
                }
            }
            from += kAgain * kThreads;
            int done = 0;  // vectors of this warp that are through
            bool again;
#pragma unroll 1
            do {
                int32_t room = kWarpRoom;
#pragma unroll 1
                for (; done < kAgain; ++done) {
                    uint4 x = v[0];
                    int32_t q = at[0];
#pragma unroll
                    for (int i = 1; i < kAgain; ++i)
                        if (done == i) {
                            x = v[i];
                            q = at[i];
                        }
                    float most = element<E>(x, 0);
#pragma unroll
                    for (int e = 1; e < kN; ++e) most = fmaxf(most, element<E>(x, e));
                    const bool hot = q >= 0 && most >= limit;
                    const uint32_t who = __ballot_sync(0xffffffffu, hot);
                    if (who == 0) continue;
                    if (__popc(who) * kN > room) break;  // the rest after a merge
                    int n = 0;
                    if (hot) {
#pragma unroll
                        for (int e = 0; e < kN; ++e) {
                            if (!(element<E>(x, e) >= limit)) continue;
                            const Key key = make_key(element<E>(x, e), (uint32_t)(sl.id0 + q * kN + e));
                            if (key > bound) {
                                put(sh, key);
                                ++n;
                            }
                        }
                    }
                    room -= __reduce_add_sync(0xffffffffu, n);
                }
                again = __syncthreads_or(done < kAgain) != 0;
                const bool full = sh.n_cand > kCand - kThreads / 32 * kWarpRoom;
                __syncthreads();
                if (full || (!again && from >= total)) {
                    merge(sh, k, tid);
                    bound = sh.bound;
                    if (bound) limit = fmaxf(limit, key_value(bound));
                }
            } while (again);
        } while (from < total);
    }
}

// A shift of the maximum in the exponent. 2^-200 is 0; a longer shift would only make the products with it
// infinite.
__device__ __forceinline__ float shift(float from, float to, float sl2)
{
    return from == -INFINITY ? 0.f : fmaxf((from - to) * sl2, -200.f);  // no values yet: the sums are 0
}

// The sums of two parts about the larger of their maxima.
__device__ __forceinline__ void join_stats(float& m, float& s, float& w, float m2, float s2, float w2, float sl2)
{
    const float mn = fmaxf(m, m2);
    const float d1 = shift(m, mn, sl2), d2 = shift(m2, mn, sl2);
    const float a1 = ex2(d1), a2 = ex2(d2);
    w = (w + d1 * s) * a1 + (w2 + d2 * s2) * a2;
    s = s * a1 + s2 * a2;
    m = mn;
}

template <typename E>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) token_logprobs_kernel(const LogprobsParams p)
{
    constexpr int kN = 32 / sizeof(E);  // elements of a sector
    constexpr int kSecs = kElems / kN;  // sectors per thread and step
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const int32_t row = blockIdx.y;
    const int32_t k = p.k;
    const E* r = static_cast<const E*>(p.logits) + row * p.row_stride;
    // The row in sectors of 32 bytes, counted from the boundary at or before its first element. This CTA's are
    // [q0, q0 + nq); those at the row's ends that hold other elements too ([0, whole0) and [whole1, nq)) are read
    // element by element. Offsets within the slice fit 32 bits.
    const int32_t mis = (int32_t)((reinterpret_cast<uintptr_t>(r) & 31) / sizeof(E));
    const int64_t secs = ((int64_t)p.V + mis + kN - 1) / kN;
    const int64_t q0 = secs * blockIdx.x / p.slices;
    const int32_t nq = (int32_t)(secs * (blockIdx.x + 1) / p.slices - q0);
    const int32_t whole0 = q0 == 0 && mis ? 1 : 0;
    const int32_t whole1 = q0 + nq == secs && (p.V + mis) % kN ? nq - 1 : nq;
    const E* base = r + (q0 * kN - mis);
    const int32_t id0 = (int32_t)(q0 * kN) - mis;  // id of the slice's first element
    const float sl2 = kLog2e / p.temperature;
    if (tid == 0) {
        sh.n_kept = sh.n_cand = 0;
        sh.bound = 0;
    }
    // a given token's logit, fetched while the row streams
    int32_t tok = -1;
    float tok_x = 0.f;
    if (tid < p.m) {
        tok = __ldg(p.tokens + (int64_t)row * p.m + tid);
        if (tok >= 0 && tok < p.V)
            tok_x = sizeof(E) == 2 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(r)[tok])
                                   : reinterpret_cast<const float*>(r)[tok];
    }
    __syncthreads();

    // The elements of those vectors at the ends: one of a thread's first few.
    bool has_edge = false;
    float edge_x = -INFINITY;
    int32_t edge_id = 0;
    if (tid < 2 * kN && nq > 0) {
        const bool tail = tid >= kN;
        const bool here = tail ? whole1 < nq && nq - 1 >= whole0 : whole0 > 0;
        const int64_t id = (q0 + (tail ? nq - 1 : 0)) * kN - mis + tid % kN;
        has_edge = here && id >= 0 && id < p.V;
        if (has_edge) {
            edge_id = (int32_t)id;
            edge_x = sizeof(E) == 2 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(r)[id])
                                    : reinterpret_cast<const float*>(r)[id];
        }
    }

    // Sectors that are not the slice's count as -inf.
    auto fetch = [&](int32_t at, uint4 (&raw)[2 * kSecs]) {
        const bool all = at >= whole0 && at + kSecs * kThreads <= whole1;
#pragma unroll
        for (int u = 0; u < kSecs; ++u) {
            const int32_t q = at + u * kThreads + tid;
            const uint32_t none = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
            if (all || (q >= whole0 && q < whole1)) {
                const uint4* src = reinterpret_cast<const uint4*>(base) + 2 * (int64_t)q;
                raw[2 * u] = __ldcs(src);
                raw[2 * u + 1] = __ldcs(src + 1);
            } else {
                raw[2 * u] = raw[2 * u + 1] = make_uint4(none, none, none, none);
            }
        }
    };
    auto value = [&](const uint4 (&raw)[2 * kSecs], int i) -> float {
        return element<E>(raw[i / (kN / 2)], i % (kN / 2));
    };
    auto step_max = [&](const uint4 (&raw)[2 * kSecs]) -> float {
        if (sizeof(E) == 2) {
            // pairs of bf16 as they lie
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw[0]);
            __nv_bfloat162 x = h[0];
#pragma unroll
            for (int i = 1; i < kElems / 2; ++i) x = __hmax2(x, h[i]);
            return fmaxf(__low2float(x), __high2float(x));
        }
        float x = value(raw, 0);
#pragma unroll
        for (int i = 1; i < kElems; ++i) x = fmaxf(x, value(raw, i));
        return x;
    };

    float m = -INFINITY, s = 0.f, w = 0.f;
    const int32_t steps = (nq + kSecs * kThreads - 1) / (kSecs * kThreads);
    const int32_t phase_len = max(1, (steps + kPhases - 1) / kPhases);
    float top = edge_x;  // the thread's largest value
    if (edge_x > -INFINITY) {
        m = edge_x;
        s = 1.f;
    }
    {
        uint4 cur[2 * kSecs], nxt[2 * kSecs];
        fetch(0, cur);
        int32_t step = 0;
#pragma unroll 1
        for (int32_t phase = 0; step < steps; ++phase) {
            const int32_t end = min(steps, step + phase_len);
            float group = -INFINITY;
#pragma unroll 1
            for (; step < end; ++step) {
                if (step + 1 < steps) fetch((step + 1) * kSecs * kThreads, nxt);
                const float mt = step_max(cur);
                group = fmaxf(group, mt);
                if (mt > m) {
                    const float d = shift(m, mt, sl2);
                    const float a = ex2(d);
                    w = (w + d * s) * a;
                    s *= a;
                    m = mt;
                }
                const float mu = m == -INFINITY ? 0.f : m;
                const uint64_t neg2 = pack2(-mu, -mu), scale2 = pack2(sl2, sl2);
                uint64_t s2 = 0, w2 = 0;
#pragma unroll
                for (int i = 0; i < kElems; i += 2) {
                    // a value of -inf has no share: 2^-200 is 0, and y stays finite for the entropy's product
                    float y0, y1;
                    unpack2(mul2(add2(pack2(value(cur, i), value(cur, i + 1)), neg2), scale2), y0, y1);
                    y0 = fmaxf(y0, -200.f);
                    y1 = fmaxf(y1, -200.f);
                    const uint64_t e2 = pack2(ex2(y0), ex2(y1));
                    s2 = add2(s2, e2);
                    w2 = fma2(pack2(y0, y1), e2, w2);
                }
                float a0, a1;
                unpack2(s2, a0, a1);
                s += a0 + a1;
                unpack2(w2, a0, a1);
                w += a0 + a1;
#pragma unroll
                for (int u = 0; u < 2 * kSecs; ++u) cur[u] = nxt[u];
            }
            sh.group[phase][tid] = __float2bfloat16_ru(group);
            top = fmaxf(top, group);
        }
    }
    if (k > 0)
        select_again<E>(sh, k, Slice{base, nq, whole0, whole1, id0, steps, phase_len}, top, has_edge, edge_x, edge_id);
    // the CTA's sums
    auto reduce_stats = [&]() {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, off), s2 = __shfl_xor_sync(0xffffffffu, s, off),
                        w2 = __shfl_xor_sync(0xffffffffu, w, off);
            join_stats(m, s, w, m2, s2, w2, sl2);
        }
        __syncthreads();
        if ((tid & 31) == 0) {
            sh.red[0][tid >> 5] = m;
            sh.red[1][tid >> 5] = s;
            sh.red[2][tid >> 5] = w;
        }
        __syncthreads();
        m = -INFINITY;
        s = w = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) join_stats(m, s, w, sh.red[0][i], sh.red[1][i], sh.red[2][i], sl2);
    };
    reduce_stats();

    if (p.slices > 1) {
        const int64_t part = (int64_t)row * p.slices + blockIdx.x;
        if (tid == 0) {
            float* st = p.part_stat + part * 4;
            st[0] = m;
            st[1] = s;
            st[2] = w;
        }
        if (tid < k) p.part_key[part * k + tid] = tid < sh.n_kept ? sh.kept[tid] : 0;
        __threadfence();
        __syncthreads();
        if (tid == 0) sh.last = atomicAdd(p.counters + row, 1) == p.slices - 1;
        __syncthreads();
        if (!sh.last) return;
        __threadfence();
        m = -INFINITY;
        s = w = 0.f;
        for (int32_t i = tid; i < p.slices; i += kThreads) {
            const float* st = p.part_stat + ((int64_t)row * p.slices + i) * 4;
            join_stats(m, s, w, __ldcg(st), __ldcg(st + 1), __ldcg(st + 2), sl2);
        }
        reduce_stats();
        if (k > 0) {
            if (tid == 0) {
                sh.n_kept = 0;
                sh.bound = 0;
            }
            __syncthreads();
            const Key* keys = p.part_key + (int64_t)row * p.slices * k;
            // The slices' lists are in order, so their first keys (and, of fewer than 128 lists, their next few) give
            // a bound that leaves little more than k keys of them all; what exceeds it is merged. (Bounds from
            // keys a thread reads at stride 128 left thousands: every thread then sees one rank of all lists.)
            Key top = 0;
            if (p.slices >= kThreads) {
                for (int32_t i = tid; i < p.slices; i += kThreads) top = max(top, __ldcg(keys + (int64_t)i * k));
            } else if (tid / p.slices < k) {
                top = __ldcg(keys + (int64_t)(tid % p.slices) * k + tid / p.slices);
            }
            const Key least = bound_of(sh.warp_key, k, tid, top, Key(0));
            if (tid == 0 && least > 0) sh.bound = least - 1;  // the key itself stays in
            __syncthreads();
            // Eight keys of each list a time, until no list goes on above the bound: mostly once (1 row of 151936, k = 64:
            // 75 lists, 18.5 us in place of 24 with all of them).
            bool more = true;
            for (int32_t first = 0; first < k && more; first += 8) {
                const int32_t width = min(8, k - first), total = p.slices * width;
                bool goes_on = false;
                for (int32_t at = 0; at < total; at += 4 * kThreads) {
                    const Key bound = sh.bound;
                    Key mine[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t j = at + i * kThreads + tid, list = j / width, place = j - list * width;
                        mine[i] = j < total ? __ldcg(keys + (int64_t)list * k + first + place) : 0;
                        goes_on = goes_on || (place == width - 1 && mine[i] > bound);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (mine[i] > bound) put(sh, mine[i]);
                    const bool last = at + 4 * kThreads >= total;
                    __syncthreads();
                    const bool full = sh.n_cand > kCand - 4 * kThreads;
                    __syncthreads();
                    if (full || last) merge(sh, k, tid);
                }
                more = __syncthreads_or(goes_on) != 0;
            }
        }
        if (tid == 0) p.counters[row] = 0;
    }

    const float ln_s = logf(s);
    const bool none = m == -INFINITY;  // every token ruled out
    auto logp = [&](float x) { return none || x == -INFINITY ? -INFINITY : (x - m) / p.temperature - ln_s; };
    if (tid == 0) {
        if (p.log_z) p.log_z[row] = none ? -INFINITY : m / p.temperature + ln_s;
        if (p.entropy) p.entropy[row] = none ? 0.f : ln_s - kLn2 * (w / s);
    }
    if (tid < p.m) {
        float out = -INFINITY;
        if (tok >= 0 && tok < p.V)
            out = logp(tok_x);
        else if (tok >= p.V)
            raise_error(p.err, DFLASH_DEVERR_TOKEN_ID);
        p.token_logp[(int64_t)row * p.m + tid] = out;
    }
    if (tid < k) {
        const Key key = tid < sh.n_kept ? sh.kept[tid] : 0;  // all k are there, unless the row holds NaN
        p.top_tokens[(int64_t)row * k + tid] = key_id(key);
        p.top_logp[(int64_t)row * k + tid] = logp(key_value(key));
    }
}

}  // namespace

int32_t logprobs_slices(int32_t R, int32_t V)
{
    // One wave of CTAs, but no more than a slice per step of the row: short rows are cut into slices of one step, half
    // a step to a whole one each. A slice more costs a row some microseconds of merging.
    const int64_t wave = (int64_t)kCtasPerSm * device_sm_count();
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>(wave / R, ((int64_t)V + kSliceElems - 1) / kSliceElems));
}

cudaError_t launch_token_logprobs(const LogprobsParams& p, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.slices, (unsigned)p.R);
    if (p.dtype == DFLASH_BF16)
        token_logprobs_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
    else
        token_logprobs_kernel<float><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dflash
