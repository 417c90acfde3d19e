// Rotary positions: pairs (x, y) of a head's dims turned by angle(position, pair),
//   (x, y) -> (x c - y s, x s + y c),  c, s = gain cos, gain sin
// in fp32, rounded once to the type of x. The transposed map, which takes gradients back, is the turn by the negative
// angle (`inverse`).
//
// A thread takes one unit (8 pairs or 16 plain dims, two 16-byte accesses) of `heads` heads of one token, two heads' loads of 16 bits in
// flight at a time. A unit's 8 angles cost some 300 instructions and are worked out once for the thread's heads: as many of
// them as leave the GPU a wave of threads, and one where only latency counts. Units of pairs and of plain dims go to
// warps of their own, so that the copies do not wait for angles. Bound: the bytes, read and written once, in large calls
// (8191 tokens of 32 heads of 128 in bf16, 134 MB: 28.4 us, 4.7 TB/s), and the launch in small ones (12 us by the host's clock).
#include <algorithm>

#include "rope.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;

// Units [first, first + units) of the rows, blocks [block0, block0 + gridDim.x): the pairs' units, then the plain ones.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 4)
    rope_kernel(const RopeParams p, const RopeUnits g, const int32_t heads, const uint32_t rotary_blocks)
{
    const bool pairs = blockIdx.x < rotary_blocks;
    const uint32_t block = pairs ? blockIdx.x : blockIdx.x - rotary_blocks;
    const uint32_t units = pairs ? g.rotated : g.units - g.rotated, groups = (p.H + heads - 1) / heads;
    const int64_t id = (int64_t)block * kThreads + threadIdx.x;
    const int64_t rest = id / units;
    const int32_t u = (int32_t)(id - rest * units) + (pairs ? 0 : g.rotated);
    const int64_t n = rest / groups;
    if (n >= p.N) return;
    const int32_t h0 = (int32_t)(rest - n * groups) * heads, h1 = min(p.H, h0 + heads);
    const UnitAt at = unit_at(g, u);
    const T* x = static_cast<const T*>(p.x) + n * p.xt;
    T* out = static_cast<T*>(p.out) + n * p.ot;
    CosSin t[8];
    if (pairs) {
        const int32_t pos = __ldg(p.positions + n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t i = 8 * u + j;
            t[j] = i < g.half ? rope_turn(pos, __ldg(p.turns + i), p.gain, p.inverse != 0) : CosSin{1.f, 0.f};
        }
    }
    if constexpr (kVec) {
        constexpr int kBatch = 4 / sizeof(T);  // heads whose loads are in flight
#pragma unroll 1
        for (int32_t h = h0; h < h1; h += kBatch) {
            RawUnit<T> raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (h + i < h1) raw[i] = load_raw(x + (h + i) * p.xh, at);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (h + i >= h1) continue;
                float a[8], b[8];
                unit_values(raw[i], at, a, b);
                if (pairs) rotate8(a, b, t);
                store_unit<true>(out + (h + i) * p.oh, at, a, b);
            }
        }
    } else {
#pragma unroll 1
        for (int32_t h = h0; h < h1; ++h) {
            float a[8], b[8];
            load_unit<false>(x + h * p.xh, at, a, b);
            if (pairs) rotate8(a, b, t);
            store_unit<false>(out + h * p.oh, at, a, b);
        }
    }
}

template <typename T, bool kVec>
cudaError_t launch_typed(const RopeParams& p, cudaStream_t stream)
{
    const RopeUnits g = rope_units(p.D, p.half, p.interleaved);
    const int64_t wave = (int64_t)device_sm_count() * 512, rows = (int64_t)p.N * g.rotated;
    int32_t heads = 1;
    while (heads < p.H && heads < 16 && rows * ((p.H + 2 * heads - 1) / (2 * heads)) >= wave) heads *= 2;
    const int64_t groups = (p.H + heads - 1) / heads;
    auto blocks = [&](int64_t units) { return (unsigned)((p.N * groups * units + kThreads - 1) / kThreads); };
    const unsigned rotary = blocks(g.rotated), plain = p.in_place ? 0u : blocks(g.units - g.rotated);
    rope_kernel<T, kVec><<<rotary + plain, kThreads, 0, stream>>>(p, g, heads, rotary);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream)
{
    if (p.dtype == DFLASH_BF16)
        return p.vec ? launch_typed<__nv_bfloat16, true>(p, stream) : launch_typed<__nv_bfloat16, false>(p, stream);
    return p.vec ? launch_typed<float, true>(p, stream) : launch_typed<float, false>(p, stream);
}

}  // namespace dflash
