// Log probabilities of given tokens, entropy and the top tokens of rows of logits, in one pass.
//
//   m = max_v l_v, y_v = (l_v - m) log2(e) / temperature, s = sum_v 2^y_v, w = sum_v y_v 2^y_v
//   log_z = m / temperature + ln s,  logp(v) = (l_v - m) / temperature - ln s,  entropy = ln s - ln 2 * w / s
// Sums are taken about the running maximum, which is subtracted from the logit itself before the scaling: the
// differences stay exact to fp32 whatever the size of the logits, and a row with one likely token keeps its
// small entropy.
//
// A row is cut into slices, a CTA of 256 threads each, read in steps of four 16-byte vectors a thread with the
// next step's loads in flight. A step's values stay in registers for everything: the maximum, the sums and the
// selection.
//
// Selection. A value and its id form a 64-bit key (order-preserving image of the value above the id's
// complement), all distinct, so "the k largest keys" is the definition. A CTA keeps its k largest so far and a bound that
// every key of theirs exceeds. A step takes part only if a thread's maximum reaches the bound. If more than k
// threads do, the k-th largest of the thread maxima is a better bound (k threads hold a key above it), found by one
// sort of 256; then at most k threads, 32 values each, can hold keys above it: at most 2048 candidates
// whatever the data, which is what the buffer holds. Candidates wait in the buffer until it fills
// (or the row ends) and are merged 192 at a time with the k kept ones by a sort of 256. On usual data the bound is close
// after the first step, and later steps add a handful.
//
// Slices leave their sums and keys in the workspace; the last CTA of a row to arrive (a counter, no waiting) merges
// them the same way and writes the row.
#include <algorithm>
#include <cmath>

#include "dflash_device.cuh"
#include "tree.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;        // 16-byte vectors per thread and step
constexpr int kCtasPerSm = 4;
constexpr int kMaxK = DFLASH_MAX_TOP_K;
constexpr int kCand = kMaxK * 32;
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

struct Shared {
    Key sort[kThreads];
    Key kept[kMaxK];
    Key cand[kCand];
    Key bound;       // keys at or below it are out
    int32_t n_cand;
    int32_t last;
    float red[3][kThreads / 32];
};

// Sorts one key per thread, largest first (bitonic; neighbours within a warp by shuffles). The result is
// also left in sh.sort.
__device__ __forceinline__ Key sort256(Shared& sh, Key k, int tid)
{
#pragma unroll 1
    for (int size = 2; size <= kThreads; size <<= 1) {
        const bool down = (tid & size) == 0;  // this run is sorted largest first
#pragma unroll 1
        for (int j = size >> 1; j > 0; j >>= 1) {
            Key other;
            if (j >= 32) {
                __syncthreads();
                sh.sort[tid] = k;
                __syncthreads();
                other = sh.sort[tid ^ j];
            } else {
                other = __shfl_xor_sync(0xffffffffu, k, j);
            }
            const bool lower = (tid & j) == 0;
            k = (lower == down) ? max(k, other) : min(k, other);
        }
    }
    __syncthreads();
    sh.sort[tid] = k;
    __syncthreads();
    return k;
}

// Merges the waiting candidates into the kept keys.
__device__ __forceinline__ void merge(Shared& sh, int32_t k, int tid)
{
    const int32_t n = sh.n_cand;
#pragma unroll 1
    for (int32_t at = 0; at < n; at += kThreads - kMaxK) {
        Key key = 0;
        if (tid < kMaxK)
            key = tid < k ? sh.kept[tid] : 0;
        else if (at + tid - kMaxK < n)
            key = sh.cand[at + tid - kMaxK];
        key = sort256(sh, key, tid);
        if (tid < k) sh.kept[tid] = key;
        __syncthreads();
    }
    if (tid == 0) {
        sh.n_cand = 0;
        sh.bound = max(sh.bound, sh.kept[k - 1]);
    }
    __syncthreads();
}

// Offers N keys per thread (key_of(i), 0 for none); `top` is the largest of them.
template <int N, typename F>
__device__ __forceinline__ void offer(Shared& sh, int32_t k, int tid, Key top, F key_of)
{
    Key bound = sh.bound;
    const int32_t waiting = sh.n_cand;  // read ahead of the barrier: a faster thread may add to it after
    const int32_t hot = __syncthreads_count(top > bound);
    if (hot == 0) return;
    if (hot > k) {
        sort256(sh, top, tid);
        bound = max(bound, sh.sort[k - 1] - 1);  // the k-th largest maximum itself stays in
        if (tid == 0) sh.bound = bound;
        __syncthreads();
    }
    if (waiting + min(hot, k) * N > kCand) {
        merge(sh, k, tid);
        bound = sh.bound;
    }
    if (top > bound) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Key key = key_of(i);
            if (key > bound) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
        }
    }
    __syncthreads();
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
    constexpr int kN = 16 / sizeof(E);
    constexpr int kElems = kVecs * kN;
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const int32_t row = blockIdx.y;
    const int32_t k = p.k;
    const E* r = static_cast<const E*>(p.logits) + row * p.row_stride;
    const int32_t mis = (int32_t)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(E));
    const int64_t vecs = ((int64_t)p.V + mis + kN - 1) / kN;
    const int64_t per = (vecs + p.slices - 1) / p.slices;
    const int64_t q0 = blockIdx.x * per, q1 = min(vecs, q0 + per);
    const float sl2 = kLog2e / p.temperature;
    if (tid == 0) {
        sh.n_cand = 0;
        sh.bound = 0;
    }
    if (tid < kMaxK) sh.kept[tid] = 0;
    __syncthreads();

    // Values outside the row (the vectors at its ends are read element by element) count as -inf without a key.
    auto fetch = [&](int64_t base, uint4 (&raw)[kVecs]) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int64_t q = base + u * kThreads + tid;
            const uint32_t none = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
            raw[u] = make_uint4(none, none, none, none);
            if (q >= q1) continue;
            if (q * kN >= mis && (q + 1) * kN - mis <= p.V) {
                raw[u] = __ldcs(reinterpret_cast<const uint4*>(r + (q * kN - mis)));
            } else {
                E* part = reinterpret_cast<E*>(&raw[u]);
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    const int64_t id = q * kN - mis + e;
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
    fetch(q0, cur);
    for (int64_t base = q0; base < q1; base += kVecs * kThreads) {
        fetch(base + kVecs * kThreads, nxt);
        float mt = -INFINITY;
#pragma unroll
        for (int i = 0; i < kElems; ++i) mt = fmaxf(mt, value(cur, i));
        if (mt > m) {
            const float d = shift(m, mt, sl2);
            const float a = ex2(d);
            w = (w + d * s) * a;
            s *= a;
            m = mt;
        }
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            // a value of -inf has no share: 2^-200 is 0, and y stays finite for the entropy's product
            const float y = fmaxf((value(cur, i) - mu) * sl2, -200.f);
            const float e = ex2(y);
            s += e;
            w = fmaf(y, e, w);
        }
        if (k > 0) {
            auto id_of = [&](int i) -> int64_t { return (base + (i / kN) * kThreads + tid) * kN - mis + i % kN; };
            auto key_of = [&](int i) -> Key {
                const int64_t id = id_of(i);
                const bool in = base + (i / kN) * kThreads + tid < q1 && id >= 0 && id < p.V;
                return in ? make_key(value(cur, i), (uint32_t)id) : 0;
            };
            Key top = 0;
            // (a thread below the bound's value has no key above it: most of them, after the first steps)
            if (sh.bound == 0 || mt >= key_value(sh.bound)) {
#pragma unroll
                for (int i = 0; i < kElems; ++i) top = max(top, key_of(i));
            }
            offer<kElems>(sh, k, tid, top, key_of);
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) cur[u] = nxt[u];
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
    if (k > 0) merge(sh, k, tid);

    if (p.slices > 1) {
        const int64_t part = (int64_t)row * p.slices + blockIdx.x;
        if (tid == 0) {
            float* st = p.part_stat + part * 4;
            st[0] = m;
            st[1] = s;
            st[2] = w;
        }
        if (tid < k) p.part_key[part * k + tid] = sh.kept[tid];
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
                sh.n_cand = 0;
                sh.bound = 0;
            }
            if (tid < kMaxK) sh.kept[tid] = 0;
            __syncthreads();
            const int64_t total = (int64_t)p.slices * k;
            const Key* keys = p.part_key + (int64_t)row * total;
            for (int64_t at = 0; at < total; at += 8 * kThreads) {
                Key mine[8], top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t j = at + i * kThreads + tid;
                    mine[i] = j < total ? __ldcg(keys + j) : 0;
                    top = max(top, mine[i]);
                }
                offer<8>(sh, k, tid, top, [&](int i) { return mine[i]; });
            }
            merge(sh, k, tid);
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
        const int32_t t = __ldg(p.tokens + (int64_t)row * p.m + tid);
        float out = -INFINITY;
        if (t >= 0 && t < p.V)
            out = logp(sizeof(E) == 2 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(r)[t])
                                      : reinterpret_cast<const float*>(r)[t]);
        else if (t >= p.V)
            raise_error(p.err, DFLASH_DEVERR_TOKEN_ID);
        p.token_logp[(int64_t)row * p.m + tid] = out;
    }
    if (tid < k) {
        const Key key = sh.kept[tid];
        p.top_tokens[(int64_t)row * k + tid] = key_id(key);
        p.top_logp[(int64_t)row * k + tid] = logp(key_value(key));
    }
}

}  // namespace

int32_t logprobs_slices(int32_t R, int32_t V)
{
    // one wave of CTAs, slices of 8192 logits or more
    const int64_t want = (int64_t)kCtasPerSm * device_sm_count() / R;
    const int64_t most = ((int64_t)V + 8191) / 8192;
    return (int32_t)std::max<int64_t>(1, std::min(want, most));
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
