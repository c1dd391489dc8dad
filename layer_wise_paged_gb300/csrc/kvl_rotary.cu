// kvl_rotary.cu -- rotary positions of rows of heads, and their gradient.
//
//   a' = gain * (a cos - b sin),  b' = gain * (b cos + a sin),  angle = position * inv_freq[i]
//   inverse: sin negated (the transposed map; with gain it is the gradient, without it also
//   the inverse).
//
// Bound by HBM: each element is read and written once.  A row's cosines and sines serve all
// its heads, so a CTA takes kRowsPerCta rows, its threads first work out the rows' pairs into
// shared memory (one pair each), then stream the heads in 16-byte vectors: a thread turns VEC
// pairs, i.e. one vector (interleaved) or two (halves, n_freq elements apart), and the
// elements after the pairs are copied as vectors.
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
    int32_t rows_per_cta;
    int32_t n_sets;
    int32_t heads_end[kMaxSets];  // heads of the sets, summed
    kvl_rows src[kMaxSets], dst[kMaxSets];
    int32_t copy_rest[kMaxSets];  // the elements after the pairs have to be copied
};

// VEC elements at p, as floats and back.  VEC * element size is 8 or 16 bytes.
template <int TYPE, int VEC>
__device__ __forceinline__ void load_vec(const uint8_t *p, float (&v)[VEC])
{
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else if constexpr (VEC == 8) {
        load8<TYPE>(p, v);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        const uint32_t u[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
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

template <int TYPE, int VEC>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    constexpr int kSize = TYPE == KVL_TYPE_FLOAT ? 4 : 2;
    extern __shared__ float2 turns[];  // [rows][n_freq] (cos, sin) with the gain
    const int64_t row0 = int64_t(blockIdx.x) * a.rows_per_cta;
    const int rows = int(min(int64_t(a.rows_per_cta), a.n_rows - row0));
    for (int i = threadIdx.x; i < rows * a.n_freq; i += kThreads) {
        const int r = i / a.n_freq, f = i - r * a.n_freq;
        float2 cs = cos_sin_of(a.positions[row0 + r], a.inv_freq[f]);
        cs.x *= a.gain;
        cs.y *= a.inverse ? -a.gain : a.gain;
        turns[i] = cs;
    }
    __syncthreads();
    // an item: one vector of a head's pairs (halves: and its partner), or of its rest
    const int per_pairs = a.interleaved ? 2 * a.n_freq / VEC : a.n_freq / VEC;
    const int per_head = per_pairs + (a.head_dim - 2 * a.n_freq) / VEC;
    const int heads = a.heads_end[a.n_sets - 1];
    const int per_row = heads * per_head, total = rows * per_row;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int r = i / per_row, rest = i - r * per_row;
        int h = rest / per_head;
        const int v = rest - h * per_head;
        int s = 0;
        while (h >= a.heads_end[s]) ++s;
        if (s) h -= a.heads_end[s - 1];
        const uint8_t *x = static_cast<const uint8_t *>(a.src[s].data) + (row0 + r) * a.src[s].row_stride +
                           h * a.src[s].head_stride;
        uint8_t *y = static_cast<uint8_t *>(a.dst[s].data) + (row0 + r) * a.dst[s].row_stride +
                     h * a.dst[s].head_stride;
        if (v >= per_pairs) {
            if (!a.copy_rest[s]) continue;
            const int at = (2 * a.n_freq + (v - per_pairs) * VEC) * kSize;
            float u[VEC];
            load_vec<TYPE, VEC>(x + at, u);
            store_vec<TYPE, VEC>(y + at, u);
        } else if (a.interleaved) {
            const float2 *t = turns + r * a.n_freq + v * (VEC / 2);
            float u[VEC], w[VEC];
            load_vec<TYPE, VEC>(x + v * VEC * kSize, u);
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) {
                w[2 * k] = u[2 * k] * t[k].x - u[2 * k + 1] * t[k].y;
                w[2 * k + 1] = u[2 * k + 1] * t[k].x + u[2 * k] * t[k].y;
            }
            store_vec<TYPE, VEC>(y + v * VEC * kSize, w);
        } else {
            const float2 *t = turns + r * a.n_freq + v * VEC;
            float u[VEC], w[VEC];
            load_vec<TYPE, VEC>(x + v * VEC * kSize, u);
            load_vec<TYPE, VEC>(x + (a.n_freq + v * VEC) * kSize, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float p = u[k], q = w[k];
                u[k] = p * t[k].x - q * t[k].y;
                w[k] = q * t[k].x + p * t[k].y;
            }
            store_vec<TYPE, VEC>(y + v * VEC * kSize, u);
            store_vec<TYPE, VEC>(y + (a.n_freq + v * VEC) * kSize, w);
        }
    }
}

template <int TYPE, int VEC>
kvl_status launch_rotary(RotaryArgs &a, void *stream)
{
    // Few rows: one a CTA, so that they spread over the SMs; many: four, so that the
    // threads' first pass (one pair each) has all of them at work.
    a.rows_per_cta = a.n_rows < 1024 ? 1 : 4;
    const int64_t grid = ceil_div64(a.n_rows, a.rows_per_cta);
    rotary_kernel<TYPE, VEC><<<unsigned(grid), kThreads, size_t(a.rows_per_cta) * a.n_freq * sizeof(float2),
                               static_cast<cudaStream_t>(stream)>>>(a);
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
        a.copy_rest[i] = !same;
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
