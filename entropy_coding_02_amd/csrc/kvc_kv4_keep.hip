// kvc_kv4_keep.hip - the accepted path of each sequence's drafted tree, moved to
// the sequence's end in every pool.  A few hundred bytes a token and head: bound
// by the chain of loads (counts, path, pages, codes), so one launch serves all
// layers and every (pool, sequence, head) has a wave of its own.
//
// In place: a path rises, so path[t] >= t, and what token t of it is moved to
// is a source only of tokens before it.  A wave moves a path in order and
// loads what a store may overwrite before it.
#include "kvc_kernels.h"
#include "kvc_kv4.h"

namespace {

constexpr int kTokens = 8;  // moved at a time

template <int D, int G>
__global__ __launch_bounds__(256) void k_kv4_keep(Kv4Keep a)
{
    constexpr int NG = D / G;
    constexpr int NV = kTokens * (D / 4) / 64;           // 16-bit pieces of V a lane
    constexpr int KL = D / 32;                           // lanes of a K row, 16 bytes each
    constexpr int NP = (kTokens * 2 * NG + 63) / 64;     // parameters a lane
    const int lane = threadIdx.x & 63;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
    const uint32_t H = (uint32_t)a.pool.H, h = wave % H, bl = wave / H;
    const uint32_t b = bl % (uint32_t)a.B, l = bl / (uint32_t)a.B;
    if (l >= (uint32_t)a.n_pools) return;
    const int n = a.n_keep[b], base = a.base[b];
    if (n <= 0) return;
    const int ps = a.pool.pshift, P = 1 << ps;
    const int cap = a.max_pages << ps;
    const int32_t *const table = a.table + b * a.table_stride, *const path = a.path + b * a.path_stride;
    bool bad = base < 0 || n > a.max_path;
    for (int t0 = 0; t0 < n && !bad; t0 += 64) {  // bad: the same in all lanes
        const int t = t0 + lane;
        bool no = false;
        if (t < n) {
            const int from = path[t], before = t ? path[t - 1] : -1;
            no = from <= before || (int64_t)base + from >= cap || (int64_t)base + t >= cap;
            if (!no)
                no = (uint32_t)table[(base + from) >> ps] >= (uint64_t)a.pool.n_pages ||
                     (uint32_t)table[(base + t) >> ps] >= (uint64_t)a.pool.n_pages;
        }
        bad = __any(no);
    }
    if (bad) {
        if (h == 0 && l == 0 && lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
        return;
    }
    uint8_t *const codes = a.pools[l].codes;
    uint32_t *const params = (uint32_t *)a.pools[l].params;
    for (int t0 = 0; t0 < n; t0 += kTokens) {
        // lanes 0..7: where a token lies and where it goes (page, place in it); one that stays is left
        int from_page = -1, to_page = -1, from = 0, to = 0;
        const int mine = t0 + lane % kTokens;
        if (mine < n && path[mine] != mine) {
            from = base + path[mine], to = base + mine;
            from_page = table[from >> ps], to_page = table[to >> ps];
            from &= P - 1, to &= P - 1;
        }
        u32x4 k;
        uint32_t prm[NP];
        uint16_t v[NV];
        const int kt = lane / KL;  // K rows: token
        const int kf = __shfl(from_page, kt & 7, 64), kto = __shfl(to_page, kt & 7, 64);
        const int k_from = __shfl(from, kt & 7, 64), k_to = __shfl(to, kt & 7, 64);
        const bool k_does = kt < kTokens && kf >= 0;
        const uint32_t k_at = 16 * (lane % KL);
        if (k_does) k = *(const u32x4 *)(codes + kv4_block(a.pool, kf, 0, h) * (P * (D / 2)) + k_from * (D / 2) + k_at);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int t = (i * 64 + lane) / (D / 4), piece = (i * 64 + lane) % (D / 4);
            const int page = __shfl(from_page, t, 64), at = __shfl(from, t, 64);
            if (page >= 0)
                v[i] = *(const uint16_t *)(codes + kv4_block(a.pool, page, 1, h) * (P * (D / 2)) + at / 4 * (2 * D) + piece * 8 +
                                           at % 4 * 2);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int t = (i * 64 + lane) / (2 * NG), kv = (i * 64 + lane) / NG % 2, g = lane % NG;
            const int page = __shfl(from_page, t & 7, 64), at = __shfl(from, t & 7, 64);
            if (t < kTokens && page >= 0) prm[i] = params[(kv4_block(a.pool, page, kv, h) * NG + g) * P + at];
        }
        if (k_does) *(u32x4 *)(codes + kv4_block(a.pool, kto, 0, h) * (P * (D / 2)) + k_to * (D / 2) + k_at) = k;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int t = (i * 64 + lane) / (D / 4), piece = (i * 64 + lane) % (D / 4);
            const int page = __shfl(to_page, t, 64), at = __shfl(to, t, 64);
            if (page >= 0)
                *(uint16_t *)(codes + kv4_block(a.pool, page, 1, h) * (P * (D / 2)) + at / 4 * (2 * D) + piece * 8 + at % 4 * 2) = v[i];
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int t = (i * 64 + lane) / (2 * NG), kv = (i * 64 + lane) / NG % 2, g = lane % NG;
            const int page = __shfl(to_page, t & 7, 64), at = __shfl(to, t & 7, 64);
            if (t < kTokens && page >= 0) params[(kv4_block(a.pool, page, kv, h) * NG + g) * P + at] = prm[i];
        }
    }
}

template <int D, int G>
hipError_t keep(const Kv4Keep &a, hipStream_t s)
{
    const int64_t waves = (int64_t)a.n_pools * a.B * a.pool.H;
    k_kv4_keep<D, G><<<dim3((uint32_t)((waves + 3) / 4)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_keep(const Kv4Keep &a, hipStream_t stream)
{
    switch (a.pool.D * 1000 + a.pool.G) {
    case 64032: return keep<64, 32>(a, stream);
    case 64064: return keep<64, 64>(a, stream);
    case 128032: return keep<128, 32>(a, stream);
    case 128064: return keep<128, 64>(a, stream);
    case 128128: return keep<128, 128>(a, stream);
    case 256032: return keep<256, 32>(a, stream);
    case 256064: return keep<256, 64>(a, stream);
    default: return keep<256, 128>(a, stream);
    }
}
