// kvl_rotary.cu -- rotary positions of rows of heads, and their gradient.
//
//   a' = gain * (a cos - b sin),  b' = gain * (b cos + a sin),  angle = position * inv_freq[i]
//   inverse: sin negated (the transposed map; with gain it is the gradient, without it also
//   the inverse).
//
// Bound by HBM: each element is read and written once (32,000 rows of 64 heads, a gradient: 188 us, 6.3 TB/s).  A CTA takes tiles of a few rows, whose angles
// its threads work out into shared memory (a pair each); then a thread keeps one vector position of a
// head (16 bytes of pairs, or two such vectors n_freq elements apart, or 16 bytes of what follows the
// pairs) and walks the tile's heads, kAhead at a time, so no index is divided and enough loads are in
// flight; the first of them leave before the angles are worked out.
#include <cmath>
#include <cstring>

#include "kvl_quant.cuh"

namespace kvl {
namespace {

constexpr int kMaxSets = 4;
constexpr int kThreads = 256;

struct RotaryArgs {
    const float *inv_freq;
    const int32_t *positions;
    int64_t n_rows;
    int32_t n_freq, head_dim, interleaved, inverse;
    float gain;
    int32_t tile_rows;
    int32_t rest_vecs;  // vectors after a head's pairs that have to be copied
    bool copy_rest;     // some destination is not its source
    int32_t n_sets;
    int32_t heads_end[kMaxSets];  // heads of the sets, summed
    kvl_rows src[kMaxSets], dst[kMaxSets];
};

// VEC elements as they are in memory (16 or 8 bytes), and as floats.
template <int TYPE, int VEC>
struct RawVec {
    using type = uint4;
};
template <>
struct RawVec<KVL_TYPE_BFLOAT, 4> {
    using type = uint2;
};
template <>
struct RawVec<KVL_TYPE_HALF, 4> {
    using type = uint2;
};

template <int TYPE, int VEC>
__device__ __forceinline__ void to_floats(const typename RawVec<TYPE, VEC>::type &raw, float (&v)[VEC])
{
    const uint32_t *u = reinterpret_cast<const uint32_t *>(&raw);
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            if constexpr (TYPE == KVL_TYPE_BFLOAT) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

template <int TYPE, int VEC>
__device__ __forceinline__ void store_vec(uint8_t *p, const float (&v)[VEC])
{
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else if constexpr (VEC == 8) {
        store8<TYPE>(p, v);
    } else {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]));
    }
}

template <int TYPE, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    constexpr int kSize = TYPE == KVL_TYPE_FLOAT ? 4 : 2, kAhead = INTERLEAVED ? 4 : 2;
    using Raw = typename RawVec<TYPE, VEC>::type;
    extern __shared__ __align__(16) float turns[];  // [rows][2][n_freq]: cosines, sines, with the gain
    const int heads = a.heads_end[a.n_sets - 1];
    const int per_pairs = INTERLEAVED ? 2 * a.n_freq / VEC : a.n_freq / VEC;  // vectors (or two) of a head's pairs
    const int per_head = per_pairs + a.rest_vecs;
    const int groups = kThreads / per_head;  // heads the CTA is at side by side
    const int v = threadIdx.x % per_head, g = threadIdx.x / per_head;
    const bool pairs = v < per_pairs;
    const int at = (pairs ? v * VEC : 2 * a.n_freq + (v - per_pairs) * VEC) * kSize;
    const int far = a.n_freq * kSize;  // from a half's vector to the other half's

    for (int64_t row0 = int64_t(blockIdx.x) * a.tile_rows; row0 < a.n_rows; row0 += int64_t(gridDim.x) * a.tile_rows) {
        const int rows = int(min(int64_t(a.tile_rows), a.n_rows - row0));
        Raw u[kAhead], w[kAhead];
        uint8_t *y[kAhead];
        int turn[kAhead];
        int r = 0, h = g;  // this thread's next head of the tile
        auto load = [&]() {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                while (h >= heads && r < rows) {
                    h -= heads;
                    ++r;
                }
                y[i] = nullptr;
                if (g < groups && r < rows) {
                    int s = 0;
#pragma unroll
                    for (int k = 0; k < kMaxSets - 1; ++k) s += k < a.n_sets - 1 && h >= a.heads_end[k];
                    const int in = h - (s ? a.heads_end[s - 1] : 0);
                    const uint8_t *x = static_cast<const uint8_t *>(a.src[s].data) + (row0 + r) * a.src[s].row_stride + in * a.src[s].head_stride + at;
                    y[i] = static_cast<uint8_t *>(a.dst[s].data) + (row0 + r) * a.dst[s].row_stride + in * a.dst[s].head_stride + at;
                    turn[i] = r * 2 * a.n_freq;
                    u[i] = *reinterpret_cast<const Raw *>(x);
                    if (!INTERLEAVED && pairs) w[i] = *reinterpret_cast<const Raw *>(x + far);
                }
                h += groups;
            }
        };
        load();
        for (int t = threadIdx.x; t < rows * a.n_freq; t += kThreads) {
            const int q = t / a.n_freq, f = t - q * a.n_freq;
            const float2 cs = cos_sin_of(a.positions[row0 + q], a.inv_freq[f]);
            turns[q * 2 * a.n_freq + f] = cs.x * a.gain;
            turns[(q * 2 + 1) * a.n_freq + f] = a.inverse ? -cs.y * a.gain : cs.y * a.gain;
        }
        __syncthreads();
        while (y[0]) {  // a thread's heads come in order: none is left when the first of a turn is none
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (!y[i]) continue;
                if (!pairs) {
                    *reinterpret_cast<Raw *>(y[i]) = u[i];
                    continue;
                }
                constexpr int n = INTERLEAVED ? VEC / 2 : VEC;
                float c[n], s[n];
                if constexpr (n >= 4) {
#pragma unroll
                    for (int k = 0; k < n; k += 4) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(turns + turn[i] + v * n + k);
                        const float4 s4 = *reinterpret_cast<const float4 *>(turns + turn[i] + a.n_freq + v * n + k);
                        c[k] = c4.x; c[k + 1] = c4.y; c[k + 2] = c4.z; c[k + 3] = c4.w;
                        s[k] = s4.x; s[k + 1] = s4.y; s[k + 2] = s4.z; s[k + 3] = s4.w;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < n; ++k) {
                        c[k] = turns[turn[i] + v * n + k];
                        s[k] = turns[turn[i] + a.n_freq + v * n + k];
                    }
                }
                float p[VEC], o[VEC];
                to_floats<TYPE, VEC>(u[i], p);
                if constexpr (INTERLEAVED) {
#pragma unroll
                    for (int k = 0; k < n; ++k) {
                        o[2 * k] = p[2 * k] * c[k] - p[2 * k + 1] * s[k];
                        o[2 * k + 1] = p[2 * k + 1] * c[k] + p[2 * k] * s[k];
                    }
                    store_vec<TYPE, VEC>(y[i], o);
                } else {
                    float q[VEC];
                    to_floats<TYPE, VEC>(w[i], q);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) o[k] = p[k] * c[k] - q[k] * s[k];
                    store_vec<TYPE, VEC>(y[i], o);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) o[k] = q[k] * c[k] + p[k] * s[k];
                    store_vec<TYPE, VEC>(y[i] + far, o);
                }
            }
            load();
        }
        __syncthreads();  // the angles are free again
    }
}

template <int TYPE, int VEC>
kvl_status launch_rotary(RotaryArgs &a, void *stream)
{
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    a.rest_vecs = a.copy_rest ? (a.head_dim - 2 * a.n_freq) / VEC : 0;
    // Few rows: one a CTA, so that they spread over the SMs; many: tiles of four on a grid that fills the GPU
    // once, so that most of the threads have an angle to work out and CTAs start only once (40 heads of 128,
    // us with one / four: 7 rows 2.2 / 3.5, 600 3.4 / 3.9, 1,200 5.4 / 5.0, 5,000 20.0 / 17.1; with two 18.2,
    // with eight 18.9).
    const int64_t most = int64_t(sms) * 4;
    a.tile_rows = a.n_rows <= most ? 1 : 4;
    const int64_t tiles = ceil_div64(a.n_rows, a.tile_rows);
    const unsigned grid = unsigned(tiles < most ? tiles : most);
    const size_t smem = size_t(a.tile_rows) * 2 * a.n_freq * sizeof(float);
    if (a.interleaved)
        rotary_kernel<TYPE, VEC, true><<<grid, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
    else
        rotary_kernel<TYPE, VEC, false><<<grid, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" kvl_status kvl_rotary(const kvl_rope *rope, int64_t n_rows, int32_t head_dim, int32_t type,
                                 const int32_t *positions, int32_t n_sets, const kvl_rows *src,
                                 const kvl_rows *dst, const int32_t *n_heads, int32_t inverse, void *stream)
{
    if (!rope || !src || !dst || !n_heads || n_sets < 1 || n_sets > kMaxSets) return KVL_EINVAL;
    if (type < KVL_TYPE_BFLOAT || type > KVL_TYPE_FLOAT || rope->reserved != 0) return KVL_EINVAL;
    if (n_rows < 0 || n_rows > INT32_MAX || head_dim <= 0 || head_dim > 512 ||
        head_dim % (type == KVL_TYPE_FLOAT ? 4 : 8))
        return KVL_EINVAL;
    if (rope->n_freq <= 0 || rope->n_freq % 4 || 2 * rope->n_freq > head_dim) return KVL_EINVAL;
    if ((rope->interleaved | inverse) & ~1) return KVL_EINVAL;
    RotaryArgs a;
    std::memset(&a, 0, sizeof(a));
    int64_t heads = 0;
    for (int i = 0; i < n_sets; ++i) {
        if (n_heads[i] <= 0) return KVL_EINVAL;
        heads += n_heads[i];
        if (heads > (1 << 16)) return KVL_EINVAL;
        a.heads_end[i] = int32_t(heads);
    }
    if (n_rows == 0) return KVL_OK;
    if (!rope->inv_freq || !positions) return KVL_EINVAL;
    if (misaligned4(rope->inv_freq) || misaligned4(positions)) return KVL_EALIGN;
    for (int i = 0; i < n_sets; ++i) {
        kvl_status s = check_rows(&src[i]);
        if (!s) s = check_rows(&dst[i]);
        if (s) return s;
        const bool same = src[i].data == dst[i].data;
        if (same && (src[i].row_stride != dst[i].row_stride || src[i].head_stride != dst[i].head_stride))
            return KVL_EINVAL;
        a.src[i] = src[i];
        a.dst[i] = dst[i];
        a.copy_rest = a.copy_rest || !same;  // (in place the copy writes what is there)
    }
    a.inv_freq = rope->inv_freq;
    a.positions = positions;
    a.n_rows = n_rows;
    a.n_freq = rope->n_freq;
    a.head_dim = head_dim;
    a.interleaved = rope->interleaved;
    a.inverse = inverse;
    a.gain = rope->gain;
    a.n_sets = n_sets;
    // 16-byte vectors where the halves start on one (16-bit types: n_freq a multiple of 8;
    // then the rest after the pairs does too), 8-byte ones otherwise
    const bool wide = rope->n_freq % 8 == 0;
    if (type == KVL_TYPE_FLOAT) return launch_rotary<KVL_TYPE_FLOAT, 4>(a, stream);
    if (type == KVL_TYPE_BFLOAT)
        return wide ? launch_rotary<KVL_TYPE_BFLOAT, 8>(a, stream) : launch_rotary<KVL_TYPE_BFLOAT, 4>(a, stream);
    return wide ? launch_rotary<KVL_TYPE_HALF, 8>(a, stream) : launch_rotary<KVL_TYPE_HALF, 4>(a, stream);
}

extern "C" kvl_status kvl_rotary_frequencies(int32_t kind, double base, int32_t n_freq, double factor,
                                             double low, double high, double trained_context,
                                             int32_t scale_gain, float *inv_freq, float *gain)
{
    if (!inv_freq || n_freq <= 0 || n_freq > 256 || !(base > 0.0) || !std::isfinite(base)) return KVL_EINVAL;
    if (kind < KVL_ROPE_PLAIN || kind > KVL_ROPE_WAVELENGTH || (scale_gain & ~1)) return KVL_EINVAL;
    if (kind != KVL_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return KVL_EINVAL;
    if (kind == KVL_ROPE_BASE && n_freq < 2) return KVL_EINVAL;
    if (kind == KVL_ROPE_WAVELENGTH && (!(high > low) || !(trained_context > 0.0))) return KVL_EINVAL;
    if (kind == KVL_ROPE_BASE) base *= std::pow(factor, double(n_freq) / (n_freq - 1));
    for (int i = 0; i < n_freq; ++i) {
        double f = std::pow(base, -double(i) / n_freq);
        if (kind == KVL_ROPE_LINEAR) f /= factor;
        if (kind == KVL_ROPE_WAVELENGTH) {
            const double turns = trained_context * f / 6.283185307179586;
            double keep = (turns - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = f * keep + f / factor * (1.0 - keep);
        }
        inv_freq[i] = float(f);
    }
    if (gain)
        *gain = scale_gain && kind != KVL_ROPE_PLAIN && factor > 1.0 ? float(0.1 * std::log(factor) + 1.0) : 1.f;
    return KVL_OK;
}
