// kvc_kv4.hip - writing tokens into the resident 4-bit cache and reading them
// back.  Both are bound by memory: a row of D channels is 2D (16-bit) or 4D
// bytes outside and D/2 + 4D/G bytes in the cache.
//
// Work is cut into quads of four consecutive tokens of one head: four tokens'
// K rows and V pieces are neighbours in a page.
#include "kvc_kernels.h"
#include "kvc_kv4.h"

namespace {


template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Max over aligned runs of LANES lanes (4, 8 or 16), within a row of 16:
// neighbours and pairs by quad_perm, then mirrored halves (whose quads
// already agree).
template <int LANES>
__device__ __forceinline__ float run_max(float v)
{
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    if (LANES >= 8) v = fmaxf(v, dpp<0x141>(v));
    if (LANES >= 16) v = fmaxf(v, dpp<0x140>(v));
    return v;
}

// Eight channels as they lie in memory, and as floats.
template <int DT>
struct Eight {
    u32x4 w[DT == KVC_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *src, int64_t i, bool vec)
    {
        if (vec) {
            const u32x4 *s = (const u32x4 *)((const uint8_t *)src + i * (DT == KVC_F32 ? 4 : 2));
            w[0] = s[0];
            if (DT == KVC_F32) w[DT == KVC_F32] = s[1];
        } else if (DT == KVC_F32) {
            for (int j = 0; j < 8; ++j) w[j / 4][j % 4] = ((const uint32_t *)src)[i + j];
        } else {
            for (int j = 0; j < 4; ++j)
                w[0][j] = ((const uint16_t *)src)[i + 2 * j] | (uint32_t)((const uint16_t *)src)[i + 2 * j + 1] << 16;
        }
    }
    __device__ __forceinline__ float at(int j) const
    {
        if (DT == KVC_F32) {
            const uint32_t b = w[j / 4][j % 4];
            return __builtin_bit_cast(float, b);
        }
        const uint32_t b = w[0][j / 2 % 4];
        if (DT == KVC_F16) return kvc_h2f(j & 1 ? b >> 16 : b & 0xFFFFu);
        return __builtin_bit_cast(float, j & 1 ? b & 0xFFFF0000u : b << 16);
    }
};

// A group's extremes as a lane collects them.  0 * x is NaN where x is Inf or
// NaN, and adding it up costs one operation a channel.
struct Extremes {
    float hi = -__builtin_inff(), nlo = -__builtin_inff(), zero = 0.0f;
    __device__ __forceinline__ void take(float x)
    {
        hi = fmaxf(hi, x);
        nlo = fmaxf(nlo, -x);
        zero = __builtin_fmaf(x, 0.0f, zero);
    }
    // a group with Inf or NaN has hi = Inf; a finite x past the fp16 range counts as its border
    __device__ __forceinline__ void close()
    {
        hi = zero == 0.0f ? __builtin_amdgcn_fmed3f(hi, -65504.0f, 65504.0f) : __builtin_inff();
        nlo = __builtin_amdgcn_fmed3f(nlo, -65504.0f, 65504.0f);
    }
};

struct GroupScale {
    uint32_t bits;  // s | lo << 16
    float lo, inv;
    bool bad;
};

__device__ __forceinline__ GroupScale group_scale(float hi, float nlo)
{
    GroupScale g;
    g.bad = hi > 65504.0f;
    const float d = hi + nlo;                     // max - min, one rounding
    const uint32_t lob = kvc_f2h(-nlo), sb = kvc_f2h(d * (1.0f / 15.0f));
    g.lo = kvc_h2f(lob);
    const float s = kvc_h2f(sb);
    // 1 / s, correctly rounded: the hardware's reciprocal is within one unit in
    // the last place, and one Newton step in fused arithmetic from there rounds
    // correctly unless the divisor's significand is all ones (Markstein 1990);
    // s has 11 bits of 24.
    const float y = __builtin_amdgcn_rcpf(s);
    const float r = __builtin_fmaf(__builtin_fmaf(-s, y, 1.0f), y, y);
    g.inv = s > 0.0f ? r : 0.0f;
    g.bits = sb | (lob << 16);
    if (g.bad) {
        g.bits = 0x7E00u << 16;
        g.lo = g.inv = 0.0f;  // every code 0 (0 times Inf or NaN is NaN, which the clamp takes to 0)
    }
    return g;
}

// WIDE: x may lie past the fp16 range and counts as its border, as in the
// extremes (lo may have been rounded up to 65504 from a smaller minimum).
template <bool WIDE>
__device__ __forceinline__ uint32_t code4(float x, const GroupScale &g)
{
    if (WIDE) x = __builtin_amdgcn_fmed3f(x, -65504.0f, 65504.0f);
    const float r = __builtin_rintf((x - g.lo) * g.inv);
    return (uint32_t)fminf(fmaxf(r, 0.0f), 15.0f);
}

// The slots of a quad; a token that is past the end, skipped or out of the
// pool has slot -1.
struct Quad {
    int64_t slot[4];
    bool run;  // four consecutive slots from a multiple of four: one page, one V piece row
};

__device__ __forceinline__ Quad load_quad(const Kv4Pool &p, const int64_t *slots, int64_t t0, int64_t n, bool flag)
{
    Quad q;
    const int64_t end = p.n_pages << p.pshift;
    bool bad = false;
    for (int i = 0; i < 4; ++i) {
        int64_t s = t0 + i < n ? slots[t0 + i] : -1;
        if (s >= end) bad = true, s = -1;
        q.slot[i] = s;
    }
    if (bad && flag) kvc_flag(p.status, KVC_DEV_BAD_INDEX);
    q.run = q.slot[0] >= 0 && (q.slot[0] & 3) == 0 && q.slot[1] == q.slot[0] + 1 && q.slot[2] == q.slot[0] + 2 &&
            q.slot[3] == q.slot[0] + 3;
    return q;
}

// The 16-bit V pieces that the four lanes of one u and one half of the n's hold
// a nibble each of (i = 8u + 2c + half, c the nibble): every lane spreads its
// codes, dword q holding pieces 2q and 2q + 1 of the half's eight, the four
// are OR-ed, and lane c keeps dword c.
__device__ __forceinline__ uint32_t v_pieces(uint32_t codes, int i)
{
    const int c = i / 2 % 4;
    uint32_t d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t two = codes >> (8 * q);
        uint32_t w = ((two & 0xFu) | (two & 0xF0u) << 12) << (4 * c);
        w |= (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0x4E, 0xF, 0xF, true);  // lanes i ^ 2
        // lanes i ^ 4: i + 4 for the even quads of a row of 16, i - 4 for the odd ones
        int o = __builtin_amdgcn_update_dpp((int)w, (int)w, 0x104, 0xF, 0x5, false);
        o = __builtin_amdgcn_update_dpp(o, (int)w, 0x114, 0xF, 0xA, false);
        d[q] = w | (uint32_t)o;
    }
    const uint32_t a = c & 1 ? d[1] : d[0], b = c & 1 ? d[3] : d[2];
    return c & 2 ? b : a;
}

// A lane quantises 8 contiguous channels of one token: one K dword, or two V
// pieces; a group is G/8 neighbouring lanes.  Both halves read alike, 16 bytes
// a lane (a V half that read each piece's own channels, 2 bytes at a time, was
// bound by L1 misses: 75 us against 57 for 32768 tokens of 8 heads of 128).
template <int D, int G, int DT, int ITEMS, bool V>
__device__ __forceinline__ void append_rows(const Kv4Pool &p, const Kv4Rows &r, int64_t n, const int64_t *slots, uint32_t block)
{
    // ITEMS pieces a lane, their loads under way together
    Eight<DT> x[ITEMS];
    int64_t slot[ITEMS];
    int head[ITEMS];
    const int64_t end = p.n_pages << p.pshift;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const uint32_t item = (block * ITEMS + u) * 256 + threadIdx.x;
        const int i = item % (D / 8), tok = item / (D / 8) % 4;
        const uint32_t qh = item / (D / 2);
        head[u] = qh % p.H;
        const int64_t t = (int64_t)(qh / p.H) * 4 + tok;
        slot[u] = -1;
        if (t >= n) continue;
        slot[u] = slots[t];
        x[u].load(r.src, t * r.token_stride + head[u] * r.head_stride + 8 * i, r.vec);
    }
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const int i = threadIdx.x % (D / 8);
        if (slot[u] < 0 || slot[u] >= end) {  // the D/8 lanes of a token skip it together
            if (slot[u] >= 0 && i == 0) kvc_flag(p.status, KVC_DEV_BAD_INDEX);
            continue;
        }
        Extremes e;
        for (int j = 0; j < 8; ++j) e.take(x[u].at(j));
        e.close();
        const GroupScale g = group_scale(run_max<G / 8>(e.hi), run_max<G / 8>(e.nlo));
        uint32_t w = 0;
        for (int j = 0; j < 8; ++j) w |= code4<DT != KVC_F16>(x[u].at(j), g) << (4 * j);
        const int P = 1 << p.pshift, off = (int)(slot[u] & (P - 1));
        const int64_t blk = kv4_block(p, slot[u] >> p.pshift, V, head[u]);
        uint8_t *dst = p.codes + blk * (P * (D / 2));
        if (V) {
            const uint32_t two = v_pieces(w, i);
            const int piece = 8 * (i % 2) + 2 * (i / 2 % 4);  // the first one's n
            uint16_t *at = (uint16_t *)(dst + (off / 4) * (2 * D) + piece * (D / 8) + i / 8 * 8 + (off % 4) * 2);
            at[0] = (uint16_t)two;
            at[D / 16] = (uint16_t)(two >> 16);
        } else {
            *(uint32_t *)(dst + off * (D / 2) + 4 * ((i % 4) * (D / 32) + i / 4)) = w;
        }
        if (i % (G / 8) == 0) {
            p.params[(blk * (D / G) + i / (G / 8)) * P + off] = g.bits;
            if (g.bad) kvc_flag(p.status, KVC_DEV_NONFINITE);
        }
    }
}

// The first half of the blocks writes K, the second V; neighbouring blocks,
// which fill the same lines of parameters, run on one XCD.
template <int D, int G, int DT, int ITEMS>
__global__ __launch_bounds__(256) void k_kv4_append(Kv4Pool p, Kv4Rows k, Kv4Rows v, int64_t n, const int64_t *slots, uint32_t k_blocks)
{
    if (blockIdx.x < k_blocks)
        append_rows<D, G, DT, ITEMS, false>(p, k, n, slots, (uint32_t)xcd_block(blockIdx.x, k_blocks));
    else
        append_rows<D, G, DT, ITEMS, true>(p, v, n, slots, (uint32_t)xcd_block(blockIdx.x - k_blocks, k_blocks));
}

// Values leave past the caches (nontemporal): they are several times the codes
// that they come from and would push them out (80000 tokens of 8 heads of 128:
// 102 us, past the caches 62 with the codes in the last-level cache, 100 with
// them in memory, where a copy of as many bytes would take 81).
template <int DT>
__device__ __forceinline__ void store8(void *dst, int64_t i, bool vec, const float *y)
{
    if (DT == KVC_F32) {
        float *d = (float *)dst + i;
        if (vec) {
            typedef float f32x4 __attribute__((ext_vector_type(4)));
            __builtin_nontemporal_store(f32x4{y[0], y[1], y[2], y[3]}, (f32x4 *)d);
            __builtin_nontemporal_store(f32x4{y[4], y[5], y[6], y[7]}, (f32x4 *)(d + 4));
        } else {
            for (int j = 0; j < 8; ++j) d[j] = y[j];
        }
        return;
    }
    u32x4 w;
    for (int j = 0; j < 4; ++j) {
        float a = y[2 * j], b = y[2 * j + 1];
        if (DT == KVC_F16) {
            // a value past the fp16 range becomes its largest; NaN stays NaN
            a = a > 65504.0f ? 65504.0f : (a < -65504.0f ? -65504.0f : a);
            b = b > 65504.0f ? 65504.0f : (b < -65504.0f ? -65504.0f : b);
            w[j] = kvc_f2h2(a, b);
        } else {
            w[j] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16;
        }
    }
    uint16_t *d = (uint16_t *)dst + i;
    if (vec) {
        __builtin_nontemporal_store(w, (u32x4 *)d);
    } else {
        for (int j = 0; j < 8; ++j) d[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
    }
}

// fp32(lo + code * s): the product of a 4-bit and an 11-bit integer is exact.
__device__ __forceinline__ float value4(uint32_t code, uint32_t bits)
{
    return __builtin_fmaf((float)code, kvc_h2f(bits & 0xFFFF), kvc_h2f(bits >> 16));
}

template <int D, int G, int DT, int ITEMS>
__device__ __forceinline__ void read_k(const Kv4Pool &p, const Kv4Rows &r, int64_t n, const int64_t *slots, uint32_t block)
{
    uint32_t w[ITEMS], bits[ITEMS];
    int64_t slot[ITEMS], t[ITEMS];
    int head[ITEMS];
    const int i = threadIdx.x % (D / 8), P = 1 << p.pshift;
    const int64_t end = p.n_pages << p.pshift;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const uint32_t item = (block * ITEMS + u) * 256 + threadIdx.x, qh = item / (D / 2);
        head[u] = qh % p.H;
        t[u] = (int64_t)(qh / p.H) * 4 + item / (D / 8) % 4;
        slot[u] = t[u] < n ? slots[t[u]] : -1;
    }
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        w[u] = bits[u] = 0;
        if (slot[u] < 0 || slot[u] >= end) continue;
        const int off = (int)(slot[u] & (P - 1));
        const int64_t blk = kv4_block(p, slot[u] >> p.pshift, 0, head[u]);
        w[u] = *(const uint32_t *)(p.codes + blk * (P * (D / 2)) + off * (D / 2) + 4 * ((i % 4) * (D / 32) + i / 4));
        bits[u] = p.params[(blk * (D / G) + i / (G / 8)) * P + off];
    }
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        if (t[u] >= n) continue;
        if (slot[u] >= end && i == 0) kvc_flag(p.status, KVC_DEV_BAD_INDEX);
        float y[8];
        for (int j = 0; j < 8; ++j) y[j] = value4(w[u] >> (4 * j) & 15, bits[u]);
        store8<DT>(r.dst, t[u] * r.token_stride + head[u] * r.head_stride + 8 * i, r.vec, y);
    }
}

// A lane writes channels 8i .. 8i + 7 of the quad's four tokens: one nibble of
// the pieces n = 8 (i % 2) .. + 7, which its neighbours read too (from L1).
template <int D, int G, int DT>
__device__ __forceinline__ void read_v(const Kv4Pool &p, const Kv4Rows &r, int64_t n, const int64_t *slots, uint32_t item)
{
    const int i = item % (D / 8);
    const uint32_t qh = item / (D / 8);
    const int head = qh % p.H;
    const int64_t t0 = (int64_t)(qh / p.H) * 4;
    if (t0 >= n) return;
    const Quad q = load_quad(p, slots, t0, n, i == 0);
    const int c = i / 2, u = c / 4, sh = 4 * (c % 4), grp = 8 * i / G;
    const int P = 1 << p.pshift;
    const int in_piece = 8 * (i % 2) * (D / 8) + u * 8;
    uint32_t w[4][8], bits[4];
    if (q.run) {
        const int off = (int)(q.slot[0] & (P - 1));
        const int64_t blk = kv4_block(p, q.slot[0] >> p.pshift, 1, head);
        const uint8_t *src = p.codes + blk * (P * (D / 2)) + (off / 4) * (2 * D) + in_piece;
        for (int j = 0; j < 8; ++j) {
            const u32x2 d = *(const u32x2 *)(src + j * (D / 8));
            for (int k = 0; k < 4; ++k) w[k][j] = d[k / 2] >> (16 * (k & 1) + sh) & 15;
        }
        const u32x4 b = *(const u32x4 *)(p.params + (blk * (D / G) + grp) * P + off);
        for (int k = 0; k < 4; ++k) bits[k] = b[k];
    } else {
        for (int k = 0; k < 4; ++k) {
            bits[k] = 0;
            for (int j = 0; j < 8; ++j) w[k][j] = 0;
            if (q.slot[k] < 0) continue;
            const int off = (int)(q.slot[k] & (P - 1));
            const int64_t blk = kv4_block(p, q.slot[k] >> p.pshift, 1, head);
            const uint8_t *src = p.codes + blk * (P * (D / 2)) + (off / 4) * (2 * D) + in_piece + (off % 4) * 2;
            for (int j = 0; j < 8; ++j) w[k][j] = *(const uint16_t *)(src + j * (D / 8)) >> sh & 15;
            bits[k] = p.params[(blk * (D / G) + grp) * P + off];
        }
    }
    for (int k = 0; k < 4; ++k) {
        if (t0 + k >= n) break;
        float y[8];
        for (int j = 0; j < 8; ++j) y[j] = value4(w[k][j], bits[k]);
        store8<DT>(r.dst, (t0 + k) * r.token_stride + head * r.head_stride + 8 * i, r.vec, y);
    }
}

template <int D, int G, int DT, int ITEMS>
__global__ __launch_bounds__(256) void k_kv4_read(Kv4Pool p, Kv4Rows k, Kv4Rows v, int64_t n, const int64_t *slots, uint32_t k_blocks)
{
    if (blockIdx.x < k_blocks)
        read_k<D, G, DT, ITEMS>(p, k, n, slots, (uint32_t)xcd_block(blockIdx.x, k_blocks));
    else
        read_v<D, G, DT>(p, v, n, slots, (uint32_t)xcd_block(blockIdx.x - k_blocks, gridDim.x - k_blocks) * 256 + threadIdx.x);
}

template <int D, int G>
hipError_t move_rows(bool append, const Kv4Pool &p, const Kv4Rows &k, const Kv4Rows &v, int64_t n, int dt,
                     const int64_t *slots, hipStream_t s)
{
    const uint32_t qh = (uint32_t)((n + 3) / 4 * p.H);
    // One piece a lane while the chip is not full (64 tokens: 2.9 us, with two
    // 3.4), two beyond (32768 tokens of 8 heads: 44 us, with one 57, four 44).
    const int items = qh * (D / 2) > 256u * 2048u ? 2 : 1;
    const uint32_t per = 256 * items;
    const uint32_t kb = append || k.dst ? (qh * (D / 2) + per - 1) / per : 0;
    const uint32_t vb = append ? kb : (v.dst ? (qh * (D / 8) + 255) / 256 : 0);
    const dim3 grid(kb + vb), block(256);
#define KV4_ITEMS(KERNEL, DT)                                                                        \
    if (items == 2) KERNEL<D, G, DT, 2><<<grid, block, 0, s>>>(p, k, v, n, slots, kb);               \
    else KERNEL<D, G, DT, 1><<<grid, block, 0, s>>>(p, k, v, n, slots, kb);
#define KV4_CASE(KERNEL)                                                                             \
    if (dt == KVC_F16) { KV4_ITEMS(KERNEL, KVC_F16) }                                                \
    else if (dt == KVC_BF16) { KV4_ITEMS(KERNEL, KVC_BF16) }                                         \
    else { KV4_ITEMS(KERNEL, KVC_F32) }
    if (append) { KV4_CASE(k_kv4_append) } else { KV4_CASE(k_kv4_read) }
#undef KV4_CASE
#undef KV4_ITEMS
    return hipGetLastError();
}

hipError_t move_piece(bool append, const Kv4Pool &p, const Kv4Rows &k, const Kv4Rows &v, int64_t n, int dt,
                      const int64_t *slots, hipStream_t s)
{
    switch (p.D * 1000 + p.G) {
    case 64032: return move_rows<64, 32>(append, p, k, v, n, dt, slots, s);
    case 64064: return move_rows<64, 64>(append, p, k, v, n, dt, slots, s);
    case 128032: return move_rows<128, 32>(append, p, k, v, n, dt, slots, s);
    case 128064: return move_rows<128, 64>(append, p, k, v, n, dt, slots, s);
    case 128128: return move_rows<128, 128>(append, p, k, v, n, dt, slots, s);
    case 256032: return move_rows<256, 32>(append, p, k, v, n, dt, slots, s);
    case 256064: return move_rows<256, 64>(append, p, k, v, n, dt, slots, s);
    default: return move_rows<256, 128>(append, p, k, v, n, dt, slots, s);
    }
}

// Rows from token t on.
Kv4Rows rows_from(Kv4Rows r, int64_t t, int dt)
{
    const int64_t off = t * r.token_stride * (dt == KVC_F32 ? 4 : 2);
    if (r.src) r.src = (const char *)r.src + off;
    if (r.dst) r.dst = (char *)r.dst + off;
    return r;
}

// A launch holds fewer than 2^32 threads, n/4 * H * D/2 for K and as many for V;
// more tokens than that take several.
hipError_t move_any(bool append, const Kv4Pool &p, const Kv4Rows &k, const Kv4Rows &v, int64_t n, int dt,
                    const int64_t *slots, hipStream_t s)
{
    const int64_t most = ((int64_t)1 << 30) / ((int64_t)p.H * (p.D / 2)) * 4;
    for (int64_t t = 0; t < n; t += most) {
        const hipError_t e = move_piece(append, p, rows_from(k, t, dt), rows_from(v, t, dt),
                                        n - t < most ? n - t : most, dt, slots + t, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, int64_t n_tokens,
                             int dtype, const int64_t *slots, hipStream_t stream)
{
    return move_any(true, pool, k, v, n_tokens, dtype, slots, stream);
}

hipError_t launch_kv4_read(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, int64_t n_tokens,
                           int dtype, const int64_t *slots, hipStream_t stream)
{
    return move_any(false, pool, k, v, n_tokens, dtype, slots, stream);
}
