// kvl_weigh_rows.cu -- the weight that few rows a sequence give each cached token.
//
// Each K byte is read once and V not at all, so what counts is bytes in flight.  A warp takes a group of 16 tokens
// through all KV heads, so that a group's sum stays in its registers and has one writer: S^T [16 tokens x 8 rows]
// = K [16 x d] Q^T with 16 x 8 x 16 tensor instructions, codes converted in registers (as attention of few rows
// does), weights by one exponential each, summed over the columns.  K comes through the warp's own ring of tiles
// (16 tokens of two heads, whose products are independent chains) by 16-byte asynchronous copies.  The rows' Q of all heads is held in shared memory; more
// rows than a tile, or more heads than fit, take further passes over the groups.
//
// Work: the groups of all entries in a row are cut into equal contiguous shares, one a CTA.
#include "kvl_weigh.cuh"

namespace kvl {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kPair = 2;         // heads of a tile (one: 256 ragged sequences 147 us, two 136)
constexpr int kStages = 2;       // tiles of a warp's ring (3 at d = 64: the same; of one head 3: the same, 6: 198 us)
constexpr int kCtasPerSm = 2;
constexpr int kQBytes = 40 * 1024;

template <int D, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kHead = kGroup * D;
    static constexpr int kTile = kPair * kHead;
    static constexpr int kHeadBytes = kRows * (D * 2 + 8);  // Q of a head, and (factor, offset) of its rows
    static constexpr int kSmem = kQBytes + kWarps * kStages * kTile;
};

// Groups [g0, g0 + groups) of an entry hold the tokens that some row sees.
__device__ __forceinline__ Cost groups_of(const WeighArgs &w, int i, void *rep)
{
    const AttendArgs &a = w.t;
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup;
    Cost c;
    c.e = load_entry(a.seqs, B, i, rep);
    if (c.e.len > w.tokens) {
        report(rep, KVL_ERANGE, i);
        c.e.len = c.e.fresh = 0;
    }
    c.tiles = 1;
    c.g0 = group_of(first_seen(a, c.e.len - c.e.fresh), B, per_block);
    c.groups = c.e.fresh > 0 && c.e.len > 0 ? group_of(c.e.len - 1, B, per_block) + 1 - c.g0 : 0;
    return c;
}

__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int CODE, int TYPE, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) weigh_rows_kernel(const __grid_constant__ WeighArgs w)
{
    using S = Shape<D, NT>;
    constexpr int kRows = S::kRows, kChunks = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_scan[kWarps];
    __shared__ uint32_t s_off;
    __shared__ int s_entry;
    __shared__ float s_scale[kWarps][kStages * kPair];
    const AttendArgs &a = w.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nn = lane >> 2, kk = lane & 3;
    const int H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int G = a.attn.n_heads / H, per_block = (B + kGroup - 1) / kGroup;
    const int64_t N = a.cache.pool_blocks, plane = int64_t(a.layer) * 2 * N;

    // ---- this CTA's share of the groups
    const int n_seq = a.seqs.n_seq, per_thread = (n_seq + kThreads - 1) / kThreads;
    const int i0 = min(n_seq, tid * per_thread), i1 = min(n_seq, i0 + per_thread);
    uint64_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += groups_of(w, i, blockIdx.x == 0 ? a.report : nullptr).groups;
    uint64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    uint64_t before = scan - mine, total = 0;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
        if (x < warp) before += s_scan[x];
        total += s_scan[x];
    }
    if (total == 0 || total >= kMostUnits) {
        if (total && blockIdx.x == 0 && tid == 0) report(a.report, KVL_ERANGE, n_seq);
        return;
    }
    const Cut cut(uint32_t(total), min(gridDim.x, (uint32_t(total) + kWarps - 1) / kWarps));
    if (blockIdx.x >= cut.shares) return;
    uint32_t u = cut.start(blockIdx.x);
    const uint32_t u_end = cut.start(blockIdx.x + 1);
    if (u >= before && u < before + mine) {
        uint32_t off = uint32_t(u - before);
        int i = i0;
        for (;; ++i) {
            const uint32_t n = groups_of(w, i, nullptr).groups;
            if (off < n) break;
            off -= n;
        }
        s_entry = i;
        s_off = off;
    }
    __syncthreads();
    int entry = s_entry;
    uint32_t off = s_off;

    __half *sq = reinterpret_cast<__half *>(smem);
    float2 *s_fb = reinterpret_cast<float2 *>(smem + w.heads_held * kRows * D * 2);
    const uint32_t ring = smem_u32(smem) + kQBytes + warp * (kStages * S::kTile);
    const uint32_t scale_at = smem_u32(&s_scale[warp][0]);
    const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
    const int row_l = lane / kChunks, ch_l = lane % kChunks, row_bytes = H * d;

    for (; u < u_end; ++entry) {
        const Cost c = groups_of(w, entry, nullptr);
        if (off >= uint32_t(c.groups)) {  // an entry of no groups
            off = 0;
            continue;
        }
        const int ga = int(off), gb = int(min(uint32_t(c.groups), off + (u_end - u)));
        u += gb - ga;
        off = 0;
        const int slot = a.seqs.slots ? a.seqs.slots[entry] : entry;
        const float *in = w.mass_in + int64_t(slot) * w.in_stride;
        float *out = w.mass_out + int64_t(slot) * w.out_stride;
        const int pos0 = c.e.len - c.e.fresh, all_rows = c.e.fresh * G;
        if (ga == 0 && in != out) {  // tokens that no row sees
            const int blk = c.g0 / per_block, past = blk * B + (c.g0 - blk * per_block) * kGroup;
            for (int j = tid; j < past; j += kThreads) out[j] = in[j];
        }
        const int count = (gb - ga - warp + kWarps - 1) / kWarps;  // groups of this warp (may be <= 0)
        for (int row_a = 0; row_a < all_rows; row_a += kRows) {
            const int rows = min(kRows, all_rows - row_a);
            const int first_pos = pos0 + row_a / G, last_pos = pos0 + (row_a + rows - 1) / G;
            const int all_hi = a.attn.causal ? min(c.e.len, first_pos + 1) : c.e.len, all_lo = first_seen(a, last_pos);
            const int any_hi = a.attn.causal ? min(c.e.len, last_pos + 1) : c.e.len, any_lo = first_seen(a, first_pos);
            int lo[NT][2], hi[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 8 * t + 2 * kk + x, pos = pos0 + (row_a + r) / G;
                    hi[t][x] = r >= rows ? 0 : a.attn.causal ? min(c.e.len, pos + 1) : c.e.len;
                    lo[t][x] = first_seen(a, pos);
                }
            for (int ha = 0; ha < H; ha += w.heads_held) {
                const int heads = min(w.heads_held, H - ha);
                __syncthreads();  // readers of the Q before
                // Q, scaled by a power of two into the range of a half, a warp a row; factor and offset of its scores
                for (int x = warp; x < heads * kRows; x += kWarps) {
                    const int h = x / kRows, r = x - h * kRows, row = row_a + r;
                    const bool ok = r < rows;
                    const int tok = ok ? row / G : 0, head = (ha + h) * G + (ok ? row - tok * G : 0);
                    const uint8_t *src = static_cast<const uint8_t *>(a.attn.q.data) +
                                         (int64_t(c.e.row0) + tok) * a.attn.q.row_stride + int64_t(head) * a.attn.q.head_stride;
                    float v[D / 32], amax = 0.f;
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) {
                        const int e = lane * 2 + 64 * y;
                        const uint32_t z = ok && e < d ? *reinterpret_cast<const uint32_t *>(src + 2 * e) : 0;
                        if constexpr (TYPE == KVL_TYPE_BFLOAT) {
                            v[2 * y] = __uint_as_float(z << 16);
                            v[2 * y + 1] = __uint_as_float(z & 0xffff0000u);
                        } else {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&z));
                            v[2 * y] = f.x;
                            v[2 * y + 1] = f.y;
                        }
                        amax = fmaxf(amax, fmaxf(fabsf(v[2 * y]), fabsf(v[2 * y + 1])));
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    const uint32_t ex = (__float_as_uint(amax) >> 23) & 0xffu;
                    const bool plain = ex < 2 || ex > 252;
                    const float up = plain ? 1.f : __uint_as_float((254u - ex) << 23);
                    const float down = plain ? 1.f : __uint_as_float(ex << 23);
#pragma unroll
                    for (int y = 0; y < D / 64; ++y)
                        *reinterpret_cast<__half2 *>(sq + x * D + lane * 2 + 64 * y) = __floats2half2_rn(v[2 * y] * up, v[2 * y + 1] * up);
                    if (lane == 0) {
                        // a row that is not there, or whose lse is infinite, gives nothing: an offset of -infinity
                        const float z = ok ? w.lse[(int64_t(c.e.row0) + tok) * a.attn.n_heads + head] : INFINITY;
                        s_fb[x] = make_float2(a.attn.sm_scale * kLog2e * down, isinf(z) ? -INFINITY : -z * kLog2e);
                    }
                }
                __syncthreads();
                if (count <= 0) continue;

                // ---- this warp's groups, a tile (16 tokens of a head) at a time.  Lane l looks after group l of a
                // batch of 32: its page and place.
                auto place_of = [&](int k, int &t0, int &nv) -> int32_t {
                    t0 = nv = 0;
                    const int g = ga + warp + kWarps * k;
                    if (k >= count) return -1;
                    const int blk = (c.g0 + g) / per_block, at = (c.g0 + g - blk * per_block) * kGroup;
                    t0 = blk * B + at;
                    nv = min(min(kGroup, B - at), c.e.len - t0);
                    if (nv <= 0) return -1;
                    const int32_t page = c.e.table[blk];
                    if (page < 0 || page >= N) {
                        report(a.report, KVL_ERANGE, entry);
                        return -1;
                    }
                    return page;
                };
                int t0_l, nv_l, t0_n, nv_n;
                int32_t page_l = place_of(lane, t0_l, nv_l), page_n = place_of(32 + lane, t0_n, nv_n);
                int base_k = 0;
                int load_k = 0, load_h = 0, at_stage = 0;  // the next tile to load
                auto load_tile = [&] {
                    if (load_k < count) {
                        const bool ahead = load_k - base_k >= 32;
                        const int32_t page = __shfl_sync(0xffffffffu, ahead ? page_n : page_l, load_k & 31);
                        const int t0 = __shfl_sync(0xffffffffu, ahead ? t0_n : t0_l, load_k & 31);
                        const int nv = page < 0 || t0 >= any_hi || t0 + kGroup <= any_lo ? 0 : __shfl_sync(0xffffffffu, ahead ? nv_n : nv_l, load_k & 31);
                        const int h = ha + load_h;
                        const uint8_t *src = codes + (((plane + max(page, 0)) * B + t0 % B) * H + h) * d;
#pragma unroll
                        for (int y = 0; y < kPair; ++y) {
                            const uint32_t dst = ring + at_stage * S::kTile + y * S::kHead;
                            const bool there = load_h + y < heads;
#pragma unroll
                            for (int x = 0; x < D / 32; ++x) {
                                const int r = x * (32 / kChunks) + row_l;
                                const bool ok = there && r < nv && ch_l * 16 < d;
                                copy_async16(dst + k_at<D>(r, ch_l), src + (ok ? r * row_bytes + y * d + ch_l * 16 : 0), ok);
                            }
                        }
                        if (lane < kPair && load_h + lane < heads && nv > 0)
                            copy_async4(scale_at + 4 * (at_stage * kPair + lane), a.cache.scales + (plane + page) * H + h + lane);
                        at_stage = at_stage + 1 == kStages ? 0 : at_stage + 1;
                        load_h += kPair;
                        if (load_h >= heads) {
                            load_h = 0;
                            ++load_k;
                        }
                    }
                    copy_async_commit();
                };
#pragma unroll
                for (int x = 0; x < kStages - 1; ++x) load_tile();
                int stage = 0;
                for (int k = 0; k < count; ++k) {
                    if (k - base_k == 32) {
                        base_k += 32;
                        page_l = page_n; t0_l = t0_n; nv_l = nv_n;
                        page_n = place_of(base_k + 32 + lane, t0_n, nv_n);
                    }
                    const int t0 = __shfl_sync(0xffffffffu, t0_l, k & 31), nv = __shfl_sync(0xffffffffu, nv_l, k & 31);
                    const bool there = __shfl_sync(0xffffffffu, page_l, k & 31) >= 0;
                    const bool seen = there && t0 < any_hi && t0 + kGroup > any_lo;
                    const bool whole = nv == kGroup && t0 >= all_lo && t0 + kGroup <= all_hi;
                    // lanes kk = 0 write tokens nn and nn + 8; what they hold is fetched meanwhile
                    float held[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f};
                    const bool again = row_a > 0 || ha > 0;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int j = t0 + nn + 8 * y;
                        if (kk == 0 && nn + 8 * y < nv)
                            held[y] = again ? out[j] : w.begin && j >= pos0 ? 0.f : in[j];
                    }
                    for (int h = 0; h < heads; h += kPair) {
                        load_tile();
                        copy_async_wait<kStages - 1>();
                        __syncwarp();
                        if (seen) {
                            const uint8_t *kt = smem + (ring - smem_u32(smem)) + stage * S::kTile;
                            float s[kPair][NT][4];
#pragma unroll
                            for (int y = 0; y < kPair; ++y)
#pragma unroll
                                for (int t = 0; t < NT; ++t) s[y][t][0] = s[y][t][1] = s[y][t][2] = s[y][t][3] = 0.f;
                            // (of an odd number of heads the last tile's second half is zeros: its Q is not looked at)
#pragma unroll
                            for (int i = 0; i < D / 64; ++i) {
                                const int ch = kk + 4 * i;
#pragma unroll
                                for (int y = 0; y < kPair; ++y) {
                                    if (y > 0 && h + y >= heads) continue;
                                    const uint4 ka = *reinterpret_cast<const uint4 *>(kt + y * S::kHead + k_at<D>(nn, ch));
                                    const uint4 kb = *reinterpret_cast<const uint4 *>(kt + y * S::kHead + k_at<D>(nn + 8, ch));
                                    uint32_t q[NT][8];
#pragma unroll
                                    for (int t = 0; t < NT; ++t) {
                                        const uint4 *p = reinterpret_cast<const uint4 *>(sq + ((h + y) * kRows + 8 * t + nn) * D + ch * 16);
                                        const uint4 x = p[0], z = p[1];
                                        q[t][0] = x.x; q[t][1] = x.y; q[t][2] = x.z; q[t][3] = x.w;
                                        q[t][4] = z.x; q[t][5] = z.y; q[t][6] = z.z; q[t][7] = z.w;
                                    }
                                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                                    for (int z = 0; z < 4; ++z) {
                                        uint32_t a0, a1, a2, a3;
                                        codes_of<CODE>(wa[z], a0, a2);
                                        codes_of<CODE>(wb[z], a1, a3);
#pragma unroll
                                        for (int t = 0; t < NT; ++t) mma16816(s[y][t], a0, a1, a2, a3, q[t][2 * z], q[t][2 * z + 1]);
                                    }
                                }
                            }
#pragma unroll
                            for (int y = 0; y < kPair; ++y) {
                                if (y > 0 && h + y >= heads) continue;
                                const float ks = s_scale[warp][stage * kPair + y];
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
                                    const float4 fb = *reinterpret_cast<const float4 *>(s_fb + (h + y) * kRows + 8 * t + 2 * kk);
#pragma unroll
                                    for (int x = 0; x < 4; ++x) {
                                        const float f = x & 1 ? fb.z : fb.x, b = x & 1 ? fb.w : fb.y;
                                        const int j = t0 + nn + 8 * (x >> 1);
                                        const bool hide = b == -INFINITY || (!whole && (nn + 8 * (x >> 1) >= nv || j < lo[t][x & 1] || j >= hi[t][x & 1]));
                                        const float p = exp2_of(fmaf(s[y][t][x], ks * f, b));
                                        sum[x >> 1] += hide ? 0.f : p;
                                    }
                                }
                            }
                        }
                        __syncwarp();  // the stage may be filled again
                        stage = stage + 1 == kStages ? 0 : stage + 1;
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
                        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
                        if (kk == 0 && nn + 8 * y < nv) out[t0 + nn + 8 * y] = held[y] + sum[y];
                    }
                }
                copy_async_wait<0>();
                __syncwarp();
            }
        }
        __syncthreads();
    }
}

template <int CODE, int TYPE, int D, int NT>
kvl_status launch_rows(WeighArgs w, int sms, void *stream)
{
    using S = Shape<D, NT>;
    static std::atomic<unsigned long long> ready[kMaxDevices];
    if (!allow_smem(weigh_rows_kernel<CODE, TYPE, D, NT>, ready, S::kSmem)) return KVL_ECUDA;
    const int most = kQBytes / S::kHeadBytes;
    w.heads_held = w.t.cache.n_kv_heads < most ? w.t.cache.n_kv_heads : most;
    const int ctas = sms * (2 * (S::kSmem + 2048) <= 227 * 1024 ? kCtasPerSm : 1);
    weigh_rows_kernel<CODE, TYPE, D, NT><<<ctas, kThreads, S::kSmem, static_cast<cudaStream_t>(stream)>>>(w);
    return launch_status();
}

template <int CODE, int TYPE>
kvl_status launch_rows_dim(const WeighArgs &w, int64_t most, int sms, void *stream)
{
    const int d = w.t.cache.head_dim;
    if (d <= 64) return most <= 8 ? launch_rows<CODE, TYPE, 64, 1>(w, sms, stream) : launch_rows<CODE, TYPE, 64, 2>(w, sms, stream);
    if (d <= 128) return most <= 8 ? launch_rows<CODE, TYPE, 128, 1>(w, sms, stream) : launch_rows<CODE, TYPE, 128, 2>(w, sms, stream);
    return launch_rows<CODE, TYPE, 256, 1>(w, sms, stream);
}

}  // namespace

kvl_status launch_weigh_rows(const WeighArgs &w, int64_t most, int sms, void *stream)
{
    const bool bf = w.t.attn.type == KVL_TYPE_BFLOAT;
    if (w.t.cache.code_type == KVL_CODE_FLOAT)
        return bf ? launch_rows_dim<KVL_CODE_FLOAT, KVL_TYPE_BFLOAT>(w, most, sms, stream)
                  : launch_rows_dim<KVL_CODE_FLOAT, KVL_TYPE_HALF>(w, most, sms, stream);
    return bf ? launch_rows_dim<KVL_CODE_INT, KVL_TYPE_BFLOAT>(w, most, sms, stream)
              : launch_rows_dim<KVL_CODE_INT, KVL_TYPE_HALF>(w, most, sms, stream);
}

}  // namespace kvl
