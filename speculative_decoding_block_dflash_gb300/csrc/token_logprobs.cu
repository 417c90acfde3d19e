// Log probabilities of given tokens, entropy and the top tokens of rows of logits, in one pass.
//
//   m = max_v l_v, y_v = (l_v - m) log2(e) / temperature, s = sum_v 2^y_v, w = sum_v y_v 2^y_v
//   log_z = m / temperature + ln s,  logp(v) = (l_v - m) / temperature - ln s,  entropy = ln s - ln 2 * w / s
// Sums are taken about the running maximum, which is subtracted from the logit itself before the scaling: the
// differences stay exact to fp32 whatever the size of the logits, and a row with one likely token keeps its
// small entropy.
//
// A row is cut into slices, a CTA of 128 threads each, read in steps of 16 values a thread with the next step's
// loads in flight. A step's values stay in registers for everything: the maximum, the sums and the selection.
//
// Selection. A value and its id form a 64-bit key (order-preserving image of the value above the id's
// complement), all distinct, so "the k largest keys" is the definition. A CTA keeps its k largest so far, and a bound
// that every key still in the running exceeds. A thread looks for candidates only in steps whose maximum reaches the
// bound's value, and forms keys only of the values that do. In the first step, where all do, the thread maxima give a
// bound: sorted within each warp (shuffles), the least of the four warps' ceil(k / 4)-th largest has k maxima at or above
// it. From then on the warps run on their own in rounds of 1, 2, 4, ... steps; a warp adds its candidates to the
// buffer, and at a round's end they and the kept keys are ranked against each other (a key's rank is the number of
// larger ones; no sort), the first k stay, and the bound follows. Each round doubles what has been seen, so on usual
// data it adds about k candidates, and a row has few barriers. A warp whose share of the buffer could overflow ends its
// round early: nothing but the time depends on the data. (Per-step barriers, a sort of 256 per merge and keys formed for
// every value of a warp with a candidate: 460 us for 1000 rows of 151937; barriers and ranks: 148.)
//
// Slices leave their sums and keys in the workspace; the last CTA of a row to arrive (a counter, no waiting) merges
// them the same way and writes the row.
#include <algorithm>
#include <cmath>

#include "dflash_device.cuh"
#include "tree.h"

namespace dflash {
namespace {

constexpr int kThreads = 128;
constexpr int kElems = 16;      // values per thread and step
constexpr int kCtasPerSm = 8;
constexpr int kSliceElems = 2048;  // a step: the shortest slice
constexpr int kMaxK = DFLASH_MAX_TOP_K;
constexpr int kWarpRoom = 32 * kElems;             // candidates a warp may add in a round: a step's at least
constexpr int kCand = kThreads / 32 * kWarpRoom;
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

struct Shared {
    Key keys[kMaxK + kCand];  // the kept ones, largest first, then the waiting candidates
    Key warp_key[kThreads / 32];
    Key bound;                // keys at or below it are out
    int32_t n_kept, n_cand;
    int32_t last;
    float red[3][kThreads / 32];
};

// Ranks the waiting candidates and the kept keys; the first k stay. Every thread of the CTA calls it after a barrier.
__device__ __forceinline__ void merge(Shared& sh, int32_t k, int tid)
{
    const int32_t n_cand = sh.n_cand;
    int32_t kept = sh.n_kept;
    Key* cand = sh.keys + kMaxK;
#pragma unroll 1
    for (int32_t at = 0; at < n_cand; at += kThreads - kMaxK) {
        const int32_t here = min(n_cand - at, kThreads - kMaxK);
        Key mine = 0;
        int32_t rank = 0;
        if (tid < kept) {
            mine = sh.keys[tid];
            rank = tid;
        } else if (tid >= kMaxK && tid - kMaxK < here) {
            mine = cand[at + tid - kMaxK];
            int32_t lo = 0, hi = kept;  // kept keys are in order
            while (lo < hi) {
                const int32_t mid = (lo + hi) >> 1;
                if (sh.keys[mid] > mine)
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
        if (mine && rank < k) sh.keys[rank] = mine;
        kept = min(k, kept + here);
        __syncthreads();
    }
    if (tid == 0) {
        sh.n_cand = 0;
        sh.n_kept = kept;
        if (kept == k) sh.bound = max(sh.bound, sh.keys[k - 1]);
    }
    __syncthreads();
}

// The j-th largest (from 0) of a warp's keys.
__device__ __forceinline__ Key warp_nth(Key k, int j, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
        const bool down = (lane & size) == 0;
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const Key other = __shfl_xor_sync(0xffffffffu, k, d);
            k = (((lane & d) == 0) == down) ? max(k, other) : min(k, other);
        }
    }
    return __shfl_sync(0xffffffffu, k, j);
}

// A bound from one key of each thread's (0: none), its largest: at least k keys exceed it, or it is the old one.
__device__ __forceinline__ void raise_bound(Shared& sh, int32_t k, int tid, Key top)
{
    const Key nth = warp_nth(top, (k + kThreads / 32 - 1) / (kThreads / 32) - 1, tid & 31);
    if ((tid & 31) == 0) sh.warp_key[tid >> 5] = nth;
    __syncthreads();
    if (tid == 0) {
        Key least = sh.warp_key[0];
        for (int w = 1; w < kThreads / 32; ++w) least = min(least, sh.warp_key[w]);
        if (least > 0) sh.bound = max(sh.bound, least - 1);  // the key itself stays in
    }
    __syncthreads();
}

__device__ __forceinline__ void put(Shared& sh, Key key) { sh.keys[kMaxK + atomicAdd(&sh.n_cand, 1)] = key; }

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
    constexpr int kN = 16 / sizeof(E);
    constexpr int kVecs = kElems / kN;
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const int32_t row = blockIdx.y;
    const int32_t k = p.k;
    const E* r = static_cast<const E*>(p.logits) + row * p.row_stride;
    // The row in 16-byte vectors, counted from the boundary at or before its first element. This CTA's are [q0, q1);
    // those at the row's ends that hold other elements too are read element by element. Offsets within the slice
    // fit 32 bits.
    const int32_t mis = (int32_t)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(E));
    const int64_t vecs = ((int64_t)p.V + mis + kN - 1) / kN;
    const int64_t per = (vecs + p.slices - 1) / p.slices;
    const int64_t q0 = min(vecs, blockIdx.x * per);
    const int32_t nq = (int32_t)(min(vecs, q0 + per) - q0);
    const int32_t whole0 = q0 == 0 && mis ? 1 : 0;
    const int32_t whole1 = q0 + nq == vecs && (p.V + mis) % kN ? nq - 1 : nq;
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

    // Values outside the row count as -inf without a key.
    auto fetch = [&](int32_t at, uint4 (&raw)[kVecs]) {
        const uint4* src = reinterpret_cast<const uint4*>(base) + at + tid;
        if (at >= whole0 && at + kVecs * kThreads <= whole1) {
#pragma unroll
            for (int u = 0; u < kVecs; ++u) raw[u] = __ldcs(src + u * kThreads);
            return;
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int32_t q = at + u * kThreads + tid;
            const uint32_t none = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
            raw[u] = make_uint4(none, none, none, none);
            if (q >= whole0 && q < whole1) {
                raw[u] = __ldcs(src + u * kThreads);
            } else if (q < nq) {
                E* part = reinterpret_cast<E*>(&raw[u]);
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    const int64_t id = (q0 + q) * kN - mis + e;
                    if (id >= 0 && id < p.V) part[e] = r[id];
                }
            }
        }
    };
    auto value = [&](const uint4 (&raw)[kVecs], int i) -> float {
        const uint4& v = raw[i / kN];
        const int e = i % kN;
        if (sizeof(E) == 2) {
            const uint32_t w = e / 2 == 0 ? v.x : e / 2 == 1 ? v.y : e / 2 == 2 ? v.z : v.w;
            return __uint_as_float(e % 2 ? w & 0xFFFF0000u : w << 16);
        }
        return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
    };

    float m = -INFINITY, s = 0.f, w = 0.f;
    uint4 cur[kVecs], nxt[kVecs];
    fetch(0, cur);
    int32_t at = 0;  // this warp's step
    float mq[kElems / 4], mt;
    // maxima of four values each, and of the step
    auto maxima = [&]() {
        mt = -INFINITY;
#pragma unroll
        for (int i = 0; i < kElems / 4; ++i) {
            mq[i] = fmaxf(fmaxf(value(cur, 4 * i), value(cur, 4 * i + 1)), fmaxf(value(cur, 4 * i + 2), value(cur, 4 * i + 3)));
            mt = fmaxf(mt, mq[i]);
        }
    };
    // one of the thread's keys in this step, of its largest value
    auto any_key = [&]() -> Key {
        // (a thread of nothing but -inf: the first value of its first vector that lies in the row)
        int first = 0;
#pragma unroll
        for (int i = kElems - 1; i >= 0; --i)
            if (value(cur, i) == mt && mt > -INFINITY) first = i;
        const int32_t id = id0 + (at + (first / kN) * kThreads + tid) * kN + first % kN;
        return at + tid < nq ? make_key(mt, (uint32_t)max(id, 0)) : 0;
    };
    // hands the step's keys above the bound to the buffer; how many
    auto push = [&](Key above) -> int {
        const float least = above ? key_value(above) : -INFINITY;
        int n = 0;
#pragma unroll
        for (int g = 0; g < kElems / 4; ++g) {
            if (!(mq[g] >= least)) continue;
#pragma unroll
            for (int i = 4 * g; i < 4 * g + 4; ++i)
                if (value(cur, i) >= least) {
                    const int32_t q = at + (i / kN) * kThreads + tid;
                    const int32_t id = id0 + q * kN + i % kN;
                    const bool in = (q >= whole0 && q < whole1) || (q < nq && id >= 0 && id < p.V);
                    const Key key = make_key(value(cur, i), (uint32_t)id);
                    if (in && key > above) {
                        put(sh, key);
                        ++n;
                    }
                }
        }
        return n;
    };
    Key bound = 0;
    if (k > 0) {
        maxima();
        raise_bound(sh, k, tid, any_key());
        bound = sh.bound;
    }
#pragma unroll 1
    for (int32_t len = 1;; len = min(2 * len, 1 << 20)) {
        int32_t room = kWarpRoom;
#pragma unroll 1
        for (int32_t todo = len; todo > 0 && at < nq; --todo) {
            maxima();
            if (k > 0) {
                const bool hot = at + tid < nq && (bound == 0 || mt >= key_value(bound));
                const uint32_t who = __ballot_sync(0xffffffffu, hot);
                if (who) {
                    if (__popc(who) * kElems > room) break;
                    room -= __reduce_add_sync(0xffffffffu, hot ? push(bound) : 0);
                }
            }
            at += kVecs * kThreads;
            if (at < nq) fetch(at, nxt);
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
            for (int u = 0; u < kVecs; ++u) cur[u] = nxt[u];
        }
        const bool more = __syncthreads_or(at < nq) != 0;
        if (k > 0) {
            merge(sh, k, tid);  // (ends with a barrier, past which the next candidates come)
            bound = sh.bound;
        }
        if (!more) break;
    }
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
        if (tid < k) p.part_key[part * k + tid] = tid < sh.n_kept ? sh.keys[tid] : 0;
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
            const int64_t total = (int64_t)p.slices * k;
            const Key* keys = p.part_key + (int64_t)row * total;
            // The slices' lists are in order, so their first keys (and, of fewer than 128 lists, their next few) give
            // a bound that leaves little more than k keys of them all; what exceeds it is merged. (Bounds from
            // keys a thread reads at stride 128 left thousands: every thread then sees one rank of all lists.)
            Key top = 0;
            if (p.slices >= kThreads) {
                for (int32_t i = tid; i < p.slices; i += kThreads) top = max(top, __ldcg(keys + (int64_t)i * k));
            } else if (tid / p.slices < k) {
                top = __ldcg(keys + (int64_t)(tid % p.slices) * k + tid / p.slices);
            }
            raise_bound(sh, k, tid, top);
            for (int64_t at = 0; at < total; at += 8 * kThreads) {
                const Key bound = sh.bound;
                Key mine[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t j = at + i * kThreads + tid;
                    mine[i] = j < total ? __ldcg(keys + j) : 0;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (mine[i] > bound) put(sh, mine[i]);
                const bool last = at + 8 * kThreads >= total;
                __syncthreads();
                const bool full = sh.n_cand > kCand - 8 * kThreads;
                __syncthreads();
                if (full || last) merge(sh, k, tid);
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
        const Key key = tid < sh.n_kept ? sh.keys[tid] : 0;  // all k are there, unless the row holds NaN
        p.top_tokens[(int64_t)row * k + tid] = key_id(key);
        p.top_logp[(int64_t)row * k + tid] = logp(key_value(key));
    }
}

}  // namespace

int32_t logprobs_slices(int32_t R, int32_t V)
{
    // one wave of CTAs, slices of kSliceElems logits or more; a slice more costs a row some microseconds of merging
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
