// New keys and values of ragged requests to their positions of the paged cache, the keys rotated on the way.
//
// Request b's n_b new rows go to positions L_b - n_b .. L_b - 1. A cache of the inputs' type takes the rotated row in fp32,
// rounded once: a thread per unit of a row (rope.cuh), bound by the bytes, or for few rows by the kernel's own latency.
//
// An e4m3 cache has a scale per page and KV head. After the call it is the smallest power of two s >= 2^-126 with
// |x| <= 448 s for all of the page's tokens, earlier and new: e4m3's relative step is the same at every power of two, so
// that no other scale would be more exact, and a page whose scale grows (or shrinks again, when rejected tokens are
// overwritten) is re-encoded without a loss but where values fall into e4m3's subnormals. A warp owns a (page, head, K or
// V): it reads the earlier tokens' bytes and the new tokens, reduces the largest magnitude, and encodes. Keys are rotated
// in fp32 and rounded to e4m3 directly. The angles of a page's tokens are worked out once per CTA, for the 8 heads of its
// warps, in shared memory. A page of up to 128 units of a head (16 tokens of 128 dims) is read once and held in registers
// between the two steps, a larger one is read twice. The warp of a page is found from the rows: the first new row of every page owns it.
#include <algorithm>

#include "e4m3.cuh"
#include "rope.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTable = 4096;  // pairs' angles that a CTA holds
constexpr int kKeep = 4;      // units of a page and head that a lane holds in registers

// Where pair i of row c lies in the table: neighbouring units' pairs j are neighbours, and rows are 64 bytes apart modulo a
// line, so that a warp's reads (pair j of 8 units of 4 rows) meet all banks. (Pairs one behind the other met 4 banks: 31.5 us in
// place of 29 for 9934 tokens of 8 heads of 128.)
struct TableAt {
    int32_t units, stride;
    __device__ __forceinline__ explicit TableAt(int32_t half) : units((half + 7) / 8), stride(8 * units + 8) {}
    __device__ __forceinline__ int32_t operator()(int32_t c, int32_t i) const { return c * stride + (i & 7) * units + (i >> 3); }
};

struct Owner {
    int32_t b, i, n, pos;  // request, row of its new ones, how many there are, position of row i in the cache
    bool ok;
};

// Whose row r is. A bad length or table of starts raises an error and is nobody's.
__device__ __forceinline__ Owner owner_of(const AppendParams& p, int32_t r, bool report)
{
    Owner o{0, 0, 0, 0, false};
    int32_t first, next;
    if (p.starts) {
        int32_t lo = 0, hi = p.B;  // starts[lo] <= r < starts[hi] as far as the ends are looked at
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (__ldg(p.starts + mid) <= r)
                lo = mid;
            else
                hi = mid;
        }
        o.b = lo;
        first = __ldg(p.starts + lo);
        next = __ldg(p.starts + lo + 1);
    } else {
        const int32_t per = p.N / p.B;
        o.b = r / per;
        first = o.b * per;
        next = first + per;
    }
    if (first < 0 || r < first || r >= next) return o;
    o.i = r - first;
    o.n = next - first;
    const int32_t L = __ldg(p.seq_lens + o.b);
    if (next > p.N || L < o.n || L > p.max_seq_len) {
        if (report) raise_error(p.err, DFLASH_DEVERR_SEQ_LEN);
        return o;
    }
    o.pos = L - o.n + o.i;
    o.ok = true;
    return o;
}

// A CTA's look at the table of starts: requests whose new rows are not all among the inputs', some of which no row leads to.
__device__ __forceinline__ void check_starts(const AppendParams& p)
{
    if (!p.starts || !p.err) return;
    for (int32_t b = threadIdx.x; b < p.B; b += kThreads) {
        const int32_t first = __ldg(p.starts + b), next = __ldg(p.starts + b + 1);
        if (next < first || (next > first && (first < 0 || next > p.N))) raise_error(p.err, DFLASH_DEVERR_SEQ_LEN);
    }
}

__device__ __forceinline__ int32_t page_of(const AppendParams& p, int32_t b, int32_t pos)
{
    const int32_t id = __ldg(p.page_table + (int64_t)b * p.max_pages + pos / p.page_size);
    if (id >= 0 && id < p.num_pages) return id;
    raise_error(p.err, DFLASH_DEVERR_PAGE_ID);
    return -1;
}

// ------------------------------------------------------------------------ caches of the inputs' type

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) append_same_kernel(const AppendParams p, const RopeUnits g)
{
    const bool value = blockIdx.y == 1;
    if (blockIdx.x == gridDim.x - 1) {
        if (!value) check_starts(p);
        return;
    }
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t units = value ? (p.D + 15) / 16 : g.units;
    const int64_t rest = id / units;
    const int32_t u = (int32_t)(id - rest * units);
    const int64_t r = rest / p.Hkv;
    if (r >= p.N) return;
    const int32_t h = (int32_t)(rest - r * p.Hkv);
    const T* row = value ? static_cast<const T*>(p.v) + r * p.vt + h * p.vh : static_cast<const T*>(p.k) + r * p.kt + h * p.kh;
    const UnitAt at = unit_at(value ? rope_units(p.D, 0, 0) : g, u);
    float a[8], b[8];
    load_unit<kVec>(row, at, a, b);
    const Owner o = owner_of(p, (int32_t)r, !value && u == 0 && h == 0);
    if (!o.ok) return;
    const int32_t page = page_of(p, o.b, o.pos);
    if (page < 0) return;
    if (!value && u < g.rotated) {
        const int32_t pos = p.positions ? __ldg(p.positions + r) : o.pos;
        CosSin t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t[j] = 8 * u + j < g.half ? rope_turn(pos, __ldg(p.turns + 8 * u + j), p.gain, false) : CosSin{1.f, 0.f};
        rotate8(a, b, t);
    }
    T* dst = static_cast<T*>(value ? p.v_cache : p.k_cache) + page * p.sp + (int64_t)(o.pos % p.page_size) * p.ss + h * p.sh;
    store_unit<kVec>(dst, at, a, b);
}

// --------------------------------------------------------------------------------------- e4m3 caches

// The largest magnitude of four bytes (as bits), NaNs left out.
__device__ __forceinline__ uint32_t e4m3_top(uint32_t w)
{
    const uint32_t m = w & 0x7f7f7f7fu;
    const uint32_t f = m & ~__vcmpeq4(m, 0x7f7f7f7fu);
    const uint32_t t = __vmaxu4(f, f >> 16);
    return max(t & 0xffu, (t >> 8) & 0xffu);
}

template <bool kVec>
__device__ __forceinline__ void store_unit8(uint8_t* row, const UnitAt& at, float (&a)[8], float (&b)[8], float inv)
{
    if (kVec && at.pairs) swap_pairs_out(a, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a[j] *= inv;
        b[j] *= inv;
    }
    const uint32_t x[4] = {e4m3x4(a[0], a[1], a[2], a[3]), e4m3x4(a[4], a[5], a[6], a[7]),
                           e4m3x4(b[0], b[1], b[2], b[3]), e4m3x4(b[4], b[5], b[6], b[7])};
    if constexpr (kVec) {
        *reinterpret_cast<uint2*>(row + at.a) = make_uint2(x[0], x[1]);
        *reinterpret_cast<uint2*>(row + (at.pairs ? at.a + 8 : at.b)) = make_uint2(x[2], x[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j < at.na) row[at.a + j * at.step] = (uint8_t)(x[j >> 2] >> (8 * (j & 3)));
            if (j < at.nb) row[at.b + j * at.step] = (uint8_t)(x[2 + (j >> 2)] >> (8 * (j & 3)));
        }
    }
}

// An earlier token's 16 bytes at the page's new scale: the value in fp32, then a power of two, one rounding to e4m3.
__device__ __forceinline__ uint4 reencoded(const uint4& w, float old, float inv)
{
    uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float v[4];
        e4m3_values(q[k], v);
        q[k] = e4m3x4(v[0] * old * inv, v[1] * old * inv, v[2] * old * inv, v[3] * old * inv);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

// Grid: rows in windows of `window` and a CTA for the table of starts, groups of 8 heads, K and V.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) append_e4m3_kernel(const AppendParams p, const RopeUnits gk, const int32_t window)
{
    __shared__ CosSin table[kTable];
    const bool value = blockIdx.z == 1;
    if (blockIdx.x == gridDim.x - 1) {
        if (!value && blockIdx.y == 0) check_starts(p);
        return;
    }
    const RopeUnits g = value ? rope_units(p.D, 0, 0) : gk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t h = blockIdx.y * kWarps + warp;
    const bool mine = h < p.Hkv;
    const T* x = value ? static_cast<const T*>(p.v) + h * p.vh : static_cast<const T*>(p.k) + h * p.kh;
    const int64_t xt = value ? p.vt : p.kt;
    uint8_t* cache = static_cast<uint8_t*>(value ? p.v_cache : p.k_cache) + h * p.sh;
    float* scales = (value ? p.v_scale : p.k_scale) + h;
    const TableAt at_table(g.half);
    const bool reports = blockIdx.y == 0 && !value && warp == 0;

    // Owners among the window's rows: a request's first new row, and the first of each page.
    const int32_t r0 = blockIdx.x * window;
    Owner own{0, 0, 0, 0, false};
    if (lane < window && r0 + lane < p.N) own = owner_of(p, r0 + lane, reports);
    uint32_t owners = __ballot_sync(0xffffffffu, own.ok && (own.i == 0 || own.pos % p.page_size == 0));
    while (owners) {
        const int src = __ffs(owners) - 1;
        owners &= owners - 1;
        const int32_t b = __shfl_sync(0xffffffffu, own.b, src), i0 = __shfl_sync(0xffffffffu, own.i, src),
                      n = __shfl_sync(0xffffffffu, own.n, src), pos0 = __shfl_sync(0xffffffffu, own.pos, src);
        const int32_t row0 = r0 + src, kept = pos0 % p.page_size;
        const int32_t rows = min(n - i0, p.page_size - kept);
        const int32_t page = page_of(p, b, pos0);
        if (page < 0) continue;  // (the same for the whole CTA)
        uint8_t* base = cache + page * p.sp;
        const int32_t d16 = p.D / 16;
        if constexpr (kVec) {
            // A lane holds its part of the page: every load in flight at once, beside the angles.
            const bool fits = rows * g.units <= 32 * kKeep && kept * d16 <= 32 * kKeep && rows * at_table.stride <= kTable;
            if (fits) {  // (the same for the whole CTA)
                RawUnit<T> raw[kKeep];
                uint4 w[kKeep];
                float old = 0.f, amax = 0.f;
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < kKeep; ++k) {
                    const int32_t t = lane + 32 * k, c = t / g.units, s = t / d16;
                    if (mine && t < rows * g.units) raw[k] = load_raw(x + (row0 + c) * xt, unit_at(g, t - c * g.units));
                    if (mine && t < kept * d16)
                        w[k] = *reinterpret_cast<const uint4*>(base + (int64_t)s * p.ss + (t - s * d16) * 16);
                }
                if (mine && kept > 0) old = scales[(int64_t)page * p.Hkv];
                if (g.half) {
                    __syncthreads();  // the table's last use is over
                    for (int32_t t = threadIdx.x; t < rows * g.half; t += kThreads) {
                        const int32_t c = t / g.half, i = t - c * g.half;
                        const int32_t pos = p.positions ? __ldg(p.positions + row0 + c) : pos0 + c;
                        table[at_table(c, i)] = rope_turn(pos, __ldg(p.turns + i), p.gain, false);
                    }
                    __syncthreads();
                }
                if (!mine) continue;
                auto values = [&](int k, int32_t c, int32_t u, float (&a)[8], float (&b)[8]) {
                    unit_values(raw[k], unit_at(g, u), a, b);
                    if (u < g.rotated) {
                        CosSin cs[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) cs[j] = table[at_table(c, 8 * u + j)];
                        rotate8(a, b, cs);
                    }
                };
#pragma unroll
                for (int k = 0; k < kKeep; ++k) {
                    const int32_t t = lane + 32 * k, c = t / g.units;
                    if (t < rows * g.units) {
                        float a[8], b[8];
                        values(k, c, t - c * g.units, a, b);
#pragma unroll
                        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(a[j]), fabsf(b[j])));
                    }
                    if (t < kept * d16)
                        top = max(max(max(e4m3_top(w[k].x), e4m3_top(w[k].y)), max(e4m3_top(w[k].z), e4m3_top(w[k].w))), top);
                }
                if (kept > 0) {
                    float v[4];
                    e4m3_values(top, v);
                    amax = fmaxf(amax, v[0] * old);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                const int32_t e = e4m3_exponent(amax);
                const float now = power_of_two(e), inv = power_of_two(-e);
#pragma unroll
                for (int k = 0; k < kKeep; ++k) {
                    const int32_t t = lane + 32 * k, c = t / g.units, u = t - c * g.units;
                    if (t < rows * g.units) {
                        float a[8], b[8];
                        values(k, c, u, a, b);
                        store_unit8<true>(base + (int64_t)(kept + c) * p.ss, unit_at(g, u), a, b, inv);
                    }
                    if (t < kept * d16 && now != old) {
                        const int32_t s = t / d16;
                        *reinterpret_cast<uint4*>(base + (int64_t)s * p.ss + (t - s * d16) * 16) = reencoded(w[k], old, inv);
                    }
                }
                if (lane == 0) scales[(int64_t)page * p.Hkv] = now;
                continue;
            }
        }
        const int32_t chunk = g.half ? max(1, min(rows, kTable / at_table.stride)) : rows;  // rows whose angles fit the table
        const bool once = chunk >= rows;
        float amax = 0.f;
        uint32_t top = 0;
        float old = 0.f, inv = 1.f;
        // first the largest magnitude, then the bytes
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int32_t c0 = 0; c0 < rows; c0 += chunk) {
                const int32_t c1 = min(rows, c0 + chunk);
                if (g.half && (pass == 0 || !once)) {
                    __syncthreads();  // the table's last use is over
                    for (int32_t t = threadIdx.x; t < (c1 - c0) * g.half; t += kThreads) {
                        const int32_t c = t / g.half, i = t - c * g.half;
                        const int32_t pos = p.positions ? __ldg(p.positions + row0 + c0 + c) : pos0 + c0 + c;
                        table[at_table(c, i)] = rope_turn(pos, __ldg(p.turns + i), p.gain, false);
                    }
                    __syncthreads();
                }
                if (!mine) continue;
#pragma unroll 2
                for (int32_t t = lane; t < (c1 - c0) * g.units; t += 32) {
                    const int32_t c = t / g.units, u = t - c * g.units;
                    const UnitAt at = unit_at(g, u);
                    float va[8], vb[8];
                    load_unit<kVec>(x + (row0 + c0 + c) * xt, at, va, vb);
                    if (u < g.rotated) {
                        CosSin cs[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            cs[j] = kVec || 8 * u + j < g.half ? table[at_table(c, 8 * u + j)] : CosSin{1.f, 0.f};
                        rotate8(va, vb, cs);
                    }
                    if (pass == 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(va[j]), fabsf(vb[j])));
                    } else {
                        store_unit8<kVec>(base + (int64_t)(kept + c0 + c) * p.ss, at, va, vb, inv);
                    }
                }
            }
            if (pass == 1 || !mine) continue;
            // the page's earlier tokens, 16 bytes a time
            if (kept > 0) {
                old = scales[(int64_t)page * p.Hkv];
                for (int32_t t = lane; t < kept * d16; t += 32) {
                    const int32_t s = t / d16;
                    const uint4 w = *reinterpret_cast<const uint4*>(base + (int64_t)s * p.ss + (t - s * d16) * 16);
                    top = max(max(max(e4m3_top(w.x), e4m3_top(w.y)), max(e4m3_top(w.z), e4m3_top(w.w))), top);
                }
                float v[4];
                e4m3_values(top, v);
                amax = fmaxf(amax, v[0] * old);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int32_t e = e4m3_exponent(amax);
            const float now = power_of_two(e);
            inv = power_of_two(-e);
            if (kept > 0 && now != old) {
                for (int32_t t = lane; t < kept * d16; t += 32) {
                    const int32_t s = t / d16;
                    uint4* at = reinterpret_cast<uint4*>(base + (int64_t)s * p.ss + (t - s * d16) * 16);
                    *at = reencoded(*at, old, inv);
                }
            }
            if (lane == 0) scales[(int64_t)page * p.Hkv] = now;
        }
    }
}

template <typename T, bool kVec>
cudaError_t launch_typed(const AppendParams& p, cudaStream_t stream)
{
    const RopeUnits g = rope_units(p.D, p.half, p.interleaved);
    if (!p.k_scale) {
        const int64_t threads = (int64_t)p.N * p.Hkv * std::max(g.units, (p.D + 15) / 16);  // (and a CTA for the table of starts)
        append_same_kernel<T, kVec>
            <<<dim3((unsigned)((threads + kThreads - 1) / kThreads + 1), 2), kThreads, 0, stream>>>(p, g);
        return cudaGetLastError();
    }
    // A CTA looks for owners among `window` rows. One row where there are few rows, so that every page has a CTA of its own;
    // a page's rows where there are many, as CTAs without an owner are only launched to end.
    const int32_t groups = (p.Hkv + kWarps - 1) / kWarps;
    const int64_t fair = (int64_t)p.N * groups * 2 / (4 * device_sm_count());
    const int32_t window = (int32_t)std::max<int64_t>(1, std::min<int64_t>(fair, std::min(p.page_size, 32)));
    append_e4m3_kernel<T, kVec>
        <<<dim3((unsigned)((p.N + window - 1) / window + 1), (unsigned)groups, 2), kThreads, 0, stream>>>(p, g, window);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_kv(const AppendParams& p, cudaStream_t stream)
{
    const bool vec = p.vec_k && p.vec_v;
    if (p.dtype == DFLASH_BF16)
        return vec ? launch_typed<__nv_bfloat16, true>(p, stream) : launch_typed<__nv_bfloat16, false>(p, stream);
    return vec ? launch_typed<float, true>(p, stream) : launch_typed<float, false>(p, stream);
}

}  // namespace dflash
