// kvl_quant.cuh -- what the 8-bit cache's translation units share: the device view of a
// cache and of a batch of sequences, host-side checks, problem reports, code conversion.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvl.h"
#include "kvl_internal.cuh"
#include "kvl_ptx.cuh"

namespace kvl {
namespace {

static_assert(sizeof(PlanHeader) <= KVL_REPORT_BYTES, "a report is a plan header's bytes");

constexpr float kTinyScale = 1e-30f;   // the smallest scale an append writes
constexpr float kLog2e = 1.4426950408889634f;

// Record a problem in a report (which is read like a plan's status; NULL: nothing).
__device__ __forceinline__ void report(void *r, int code, long long detail)
{
    if (r) record_error(static_cast<PlanHeader *>(r), code, static_cast<unsigned long long>(detail));
}

// One batch entry, resolved.  n = 0 for an entry that is left out.
struct Entry {
    const int32_t *table;
    int32_t len;    // tokens held, the fresh ones included
    int32_t fresh;  // fresh rows
    int32_t row0;   // first fresh row
};

__device__ __forceinline__ Entry load_entry(const kvl_sequences &s, int32_t block_tokens, int32_t i,
                                            void *rep)
{
    Entry e;
    const int32_t a = s.starts[i], b = s.starts[i + 1];
    const int32_t slot = s.slots ? s.slots[i] : i;
    e.table = nullptr;
    e.row0 = a;
    e.len = 0;
    e.fresh = 0;
    if (a < 0 || b < a || b > s.n_rows || slot < 0 || slot >= s.n_slots) {
        report(rep, KVL_EINVAL, i);
        return e;
    }
    const int32_t len = s.lens[slot];
    int64_t first, cap;
    if (s.table_offsets) {
        first = s.table_offsets[slot];
        cap = s.table_offsets[slot + 1] - first;
    } else {
        first = int64_t(slot) * s.table_stride;
        cap = s.table_stride;
    }
    if (len < 0 || ceil_div64(len, block_tokens) > cap) {
        report(rep, KVL_ERANGE, i);
        return e;
    }
    e.table = s.tables + first;
    e.len = len;
    e.fresh = b - a;
    return e;
}

// ---- host-side checks -----------------------------------------------------------------

inline kvl_status check_cache(const kvl_cache *c)
{
    if (!c || c->n_layers <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->block_tokens <= 0 ||
        c->pool_blocks <= 0 || c->pool_blocks > INT32_MAX || c->reserved != 0)
        return KVL_EINVAL;
    if (c->head_dim % 16 || c->head_dim > 256) return KVL_EINVAL;
    if (c->n_kv_heads > 4096 || c->block_tokens > (1 << 20)) return KVL_EINVAL;
    if (c->code_type != KVL_CODE_FLOAT && c->code_type != KVL_CODE_INT) return KVL_EINVAL;
    if (!c->codes || !c->scales) return KVL_EINVAL;
    if (!aligned16(c->codes) || (reinterpret_cast<uintptr_t>(c->scales) & 3u)) return KVL_EALIGN;
    return KVL_OK;
}

inline bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

inline kvl_status check_sequences(const kvl_sequences *s)
{
    if (!s || s->n_seq < 0 || s->n_slots < 0 || s->n_rows < 0 || s->n_rows > INT32_MAX) return KVL_EINVAL;
    if (s->n_seq == 0 || s->n_rows == 0) return KVL_OK;  // nothing to do, nothing to read
    if (s->n_seq > (1 << 20) || !s->tables || !s->lens || !s->starts || s->n_slots == 0) return KVL_EINVAL;
    if (!s->slots && s->n_seq > s->n_slots) return KVL_EINVAL;
    if (!s->table_offsets && (s->table_stride <= 0 || s->table_stride > INT32_MAX)) return KVL_EINVAL;
    if (misaligned4(s->tables) || misaligned4(s->lens) || misaligned4(s->slots) || misaligned4(s->starts) ||
        (reinterpret_cast<uintptr_t>(s->table_offsets) & 7u))
        return KVL_EALIGN;
    return KVL_OK;
}

inline kvl_status check_rows(const kvl_rows *r)
{
    if (!r || !r->data) return KVL_EINVAL;
    if (!aligned16(r->data) || (r->row_stride & 15) || (r->head_stride & 15)) return KVL_EALIGN;
    return KVL_OK;
}

inline bool bad_report(const void *r) { return !aligned16(r); }

// Let `kernel` use `bytes` of dynamic shared memory (cached per context, as the copy
// kernels' attribute is).
template <typename K>
inline bool allow_smem(K kernel, std::atomic<unsigned long long> (&ready)[kMaxDevices], int bytes)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    const unsigned long long ctx = current_context_id();
    if (ctx != 0 && ready[dev].load(std::memory_order_acquire) == ctx) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return false;
    ready[dev].store(ctx, std::memory_order_release);
    return true;
}

// ---- element types ---------------------------------------------------------------------

// 8 consecutive elements of a row as floats, and back (each rounded once).
template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t *p, float (&v)[8])
{
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (TYPE == KVL_TYPE_BFLOAT)
                f = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
            else
                f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    uint32_t r;
    if constexpr (TYPE == KVL_TYPE_BFLOAT) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        r = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        r = *reinterpret_cast<const uint32_t *>(&h);
    }
    return r;
}

template <int TYPE>
__device__ __forceinline__ void store8(uint8_t *p, const float (&v)[8])
{
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 w;
        w.x = pack2<TYPE>(v[0], v[1]);
        w.y = pack2<TYPE>(v[2], v[3]);
        w.z = pack2<TYPE>(v[4], v[5]);
        w.w = pack2<TYPE>(v[6], v[7]);
        *reinterpret_cast<uint4 *>(p) = w;
    }
}

// ---- codes -------------------------------------------------------------------------------

// The nearest codes (ties to even) of four values already scaled, clamped to the largest one; a NaN
// becomes the NaN code (float) or 0 (int).
template <int CODE>
__device__ __forceinline__ uint32_t to_codes4(float a, float b, float c, float d)
{
    if constexpr (CODE == KVL_CODE_FLOAT) {
        uint32_t r;
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    } else {
        auto one = [](float x) { return uint32_t(__float2int_rn(x != x ? 0.f : fminf(fmaxf(x, -127.f), 127.f))) & 0xffu; };
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    }
}

// The four codes of w as halves, two and two: exact for both code types.  An integer code c is read as
// the half 1024 + (c + 128), of which 1152 is taken.
template <int CODE>
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (CODE == KVL_CODE_FLOAT) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t x = w ^ 0x80808080u;
        const uint32_t u = __byte_perm(x, 0x64646464u, 0x5140), v = __byte_perm(x, 0x64646464u, 0x5342);
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&u), bias), b = __hsub2(*reinterpret_cast<const __half2 *>(&v), bias);
        lo = *reinterpret_cast<const uint32_t *>(&a);
        hi = *reinterpret_cast<const uint32_t *>(&b);
    }
}

// ---- rotary positions ----------------------------------------------------------------------

// cos and sin of p * f.  The angle in turns is p * (f / 2 pi); f / 2 pi is held as the sum of
// three floats, every product with p is split into its rounded value and what that leaves
// (Dekker's arithmetic), and whole turns are taken out of each term before they are added.
// So the fraction of a turn is right to a few 2^-25 for every 32-bit position, where p * f
// in one float has lost it from p = 10^5 on.
__device__ __forceinline__ float2 cos_sin_of(int32_t p, float f)
{
    constexpr float k0 = 0.15915494f, k1 = 6.4206382e-09f, k2 = 7.342739e-17f;  // sum: 1 / (2 pi)
    const float h0 = f * k0;
    const float a = fmaf(f, k0, -h0), b = f * k1;
    const float h1 = a + b;
    const float a1 = h1 - b;
    const float h2 = (a - a1) + (b - (h1 - a1)) + fmaf(f, k1, -b) + f * k2;
    const float P = float(p);
    const float rest = float(static_cast<long long>(p) - static_cast<long long>(P));  // what P has rounded away
    auto part = [](float x, float y) {  // x * y without its whole turns
        const float q = x * y, r = fmaf(x, y, -q);
        return (q - rintf(q)) + (r - rintf(r));
    };
    float turn = part(P, h0);
    if (fabsf(P) >= 16777216.f) turn += part(rest, h0) + rest * h1;
    turn += part(P, h1) + P * h2;
    float2 r;
    sincospif(2.f * turn, &r.y, &r.x);
    return r;
}

}  // namespace
}  // namespace kvl
