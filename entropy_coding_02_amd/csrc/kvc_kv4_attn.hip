// kvc_kv4_attn.hip - attention over the resident 4-bit cache.
//
// A cached value is y = lo + s n, n = 0..15.  A code within the mantissa of an
// fp16 whose exponent is zero is the subnormal n 2^-24 (or, four bits up,
// n 2^-20), exactly, and a packed multiplication makes it n 2^-9, two codes at
// a time; (s, lo) never touch the matrix operands:
//   logits   q.k = sum_g s_g (sum_{c in g} q_c n_c) + lo_g (sum_{c in g} q_c);
//            a query row is scaled by a power of two to just under 2^15 (an
//            fp16 then holds every bit of it that fp32 sums would), so the
//            products are exact;
// (The matrix instructions take the subnormals too, but align a sum's products
// by exponent, and a subnormal's leading bits lie up to ten places below its:
// outputs that average many keys then lost twice their last fp16 bit.)
//   output   o_c = sum_j (p_j s_jg) (n_jc - 7.5) + sum_j p_j mid_jg,  c in group g,
//            mid = lo + 7.5 s.  Sums of n itself are all positive and cancel
//            against lo; what they rounded off added up (2048 queries over 8192
//            keys of values of either sign: outputs off by 8e-5 in the mean,
//            centred by 8e-7, in the same time).
// p_j s_jg enters the matrix product as two fp16 terms (22 bits): one would
// be an error of the output's own size, since n s is up to twice the value it
// belongs to.  They keep those bits because p is taken relative not to the
// row's largest logit but to the largest p_j s_j, s_j the largest s of key j's
// groups, of which the product is 2^7: neither a token far larger than the others
// that the row hardly looks at, nor one far smaller that it looks at alone, takes
// the others' bits.  (Within a token a group whose s is 2^-k of the largest
// keeps 22 bits up to k = 10, and one fewer for each more.)  That maximum is let be
// until a p s passes it by 2^8: the sums are rescaled a few times a row rather
// than at every new maximum of any of a wave's rows, and p s stays below 2^15.
//
// Orientation: S^T = K q^T (16 keys x 16 query rows), so a lane holds one
// query row and four keys of a tile, which is just what P^T needs as the
// right operand of O^T = V^T P^T (keys 4h .. 4h+3 of two tiles are its eight
// k indices): probabilities never cross lanes, the terms with mid and the row
// sums are plain fp32 sums per lane, added over the four lanes of a row once
// at the end.
#include <algorithm>

#include "kv4_rows.h"

namespace {

template <int D, int G, bool BF>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : D == 128 ? (G == 32 ? 2 : 3) : 4) void k_kv4_attn(Kv4Attn a)
{
    constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = Stage<D, G>::NP, TILE = 64 * NP, NQ = (NW + kWaves - 1) / kWaves;
    // Each wave's results; while it runs, its parameters, [tile] K's s, then
    // [tile][s|mid] V's, each [group][16 keys], in fp32 (mixed-precision instructions run at half
    // rate), then [tile] log2 of each key's largest s of V.
    __shared__ __align__(16) float lds_o[kWaves][16][D];
    __shared__ float lds_ml[kWaves][2][16];
    // The query operands, which as registers would cost a wave a SIMD.
    __shared__ u32x4 lds_q[NW][64];
    Job j;
    if (!make_job<16>(a, j)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, h = lane >> 4;  // this lane's query row, and its four keys of each tile
    float *const prm = &lds_o[wave][0][0];
    static_assert(6 * TILE + 32 <= 16 * D, "the parameters fit where the results go");
    const int row = j.row0 + col, qi = row / a.R;
    const int b_end = min(j.u1 * 4, (j.kend + 31) / 32);
    int blk = j.u0 * 4 + wave;
    const bool work = blk < b_end;
    const WaveAt<D, G> wat(a, j);

    // The pages of this wave's first two blocks, and its row of q (all of it,
    // for the row's largest; every wave then stores a part of the operands).
    int32_t first[2] = {0, 0}, pages[2] = {0, 0};
    float up;  // what the lane's row of logits is to be multiplied by
    {
        u32x4 qw[NW];
        load_query<D, BF>(a, j, row, qi, h, row < j.rows, qw);
        if (work) {
            load_pages(wat, blk, first);
            load_pages(wat, blk + kWaves, pages);
        }
        const float f = scale_query<D, BF>(a, qw, up);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            u32x4 w = qw[i * kWaves];
#pragma unroll
            for (int k = 1; k < kWaves; ++k)
                if (k < NW && wave == k) w = qw[(i * kWaves + k) % NW];
            if (wave + i * kWaves < NW) lds_q[wave + i * kWaves][lane] = query_operand<BF>(w, f);
        }
        lds_barrier();
    }

    f32x4 o[NT];
    // In powers of 2: pass, the p s at which the sums are rescaled, and ref, what p is relative to.
    float z[NG], pass = -__builtin_inff(), ref = -__builtin_inff(), mu = 0.0f, l = 0.0f;
#pragma unroll
    for (int c = 0; c < NT; ++c) o[c] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < NG; ++g) z[g] = 0.0f;
    if (work) {
        const LaneAt<D, G> at(lane, a.pool);
        Stage<D, G> cur, next;
        bool bad_page = false;
        load_stage<D, G>(wat, blk, first, at, cur, bad_page);

        // the group sums of q, in the codes' unit
        float qs[NG];
        {
            const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};  // 1
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c = {0, 0, 0, 0};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) c = mfma(ones, lds_q[s][lane], c);
                qs[g] = c[0] * 0x1p-9f;
            }
        }
        const u32x4 sums = sum_operand<NG>(qs, h);
        const int pos = j.pos0 + qi;
        const int k_hi = a.causal ? min(j.len, pos + 1) : j.len;  // keys k_lo <= key < k_hi
        const int k_lo = a.window ? max(0, pos - a.window + 1) : 0;
        // keys that every row of the tile sees
        const int all_hi = a.causal ? min(j.len, j.pos0 + j.row0 / a.R + 1) : j.len;
        const int all_lo = a.window ? j.pos0 + min(j.row0 + 15, j.rows - 1) / a.R - a.window + 1 : 0;
        // A block's codes are on their way while the one before is worked on,
        // and its pages one block earlier still.  The last turns load the last
        // tile again rather than branch: where a load may or may not have been
        // issued, the wait for an older one is a wait for all.
        for (; blk < b_end; blk += kWaves) {
            int32_t after[2];  // loads return in order: before the codes, or they would wait for them
            load_pages(wat, blk + 2 * kWaves, after);
            load_stage<D, G>(wat, blk + kWaves, pages, at, next, bad_page);
            pages[0] = after[0], pages[1] = after[1];

#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    prm[t * TILE + 64 * i + lane] = s_of(cur.kp[t][i]);
                    prm[(2 * t + 2) * TILE + 64 * i + lane] = s_of(cur.vp[t][i]);
                    prm[(2 * t + 3) * TILE + 64 * i + lane] = mid_of(cur.vp[t][i]);
                }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float s = s_of(cur.vp[t][0]);
#pragma unroll
                for (int i = 1; i < NP; ++i) s = fmaxf(s, s_of(cur.vp[t][i]));
                prm[6 * TILE + 16 * t + col] = log2_top<NG>(s);
            }
            const int key0 = blk * 32;
            const bool partial = key0 + 32 > all_hi || key0 < all_lo;
            f32x4 x[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) x[t] = mfma(lo_operand<NG>(cur.kp[t], h), sums, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) {
                    const u32x4 q = lds_q[s][lane];
                    c[0] = mfma(code_octet(cur.k[0][s]), q, c[0]);
                    c[1] = mfma(code_octet(cur.k[1][s]), q, c[1]);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 ks = *(const f32x4 *)&prm[t * TILE + 16 * g + 4 * h];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[t][i] = __builtin_fmaf(ks[i], c[t][i], x[t][i]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            float mul = up;
            if (a.softcap > 0.0f) cap_logits(a.softcap, x, mul);
            if (partial)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = key0 + 16 * (i / 4) + 4 * h + i % 4;
                    if (key < k_lo || key >= k_hi) x[i / 4][i % 4] = -__builtin_inff();
                }
            float top = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 ls = *(const f32x4 *)&prm[6 * TILE + 16 * t + 4 * h];
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, __builtin_fmaf(x[t][i], mul, ls[i]));
            }
            if (__any(top > pass)) {
                const float f = rescale(top, pass, ref, mu);
                l *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) z[g] *= f;
#pragma unroll
                for (int c = 0; c < NT; ++c) o[c] *= f;
            }
            float p[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i / 4][i % 4] = exp2_fast(__builtin_fmaf(x[i / 4][i % 4], mul, -mu));
                l += p[i / 4][i % 4];
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                u32x4 hi, lo;
                f32x4 vs[2], vmid[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    vs[t] = *(const f32x4 *)&prm[(2 * t + 2) * TILE + 16 * g + 4 * h];
                    vmid[t] = *(const f32x4 *)&prm[(2 * t + 3) * TILE + 16 * g + 4 * h];
                }
                if (partial) {
                    // what lies at a key that the row does not see may be anything, NaN too
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (x[i / 4][i % 4] == -__builtin_inff()) vs[i / 4][i % 4] = vmid[i / 4][i % 4] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float s0 = vs[i / 4][i % 4], s1 = vs[i / 4][i % 4 + 1];
                    const float p0 = p[i / 4][i % 4], p1 = p[i / 4][i % 4 + 1];
                    z[g] = __builtin_fmaf(p0, vmid[i / 4][i % 4], z[g]);
                    z[g] = __builtin_fmaf(p1, vmid[i / 4][i % 4 + 1], z[g]);
                    const f32x2 a2 = {p0 * s0, p1 * s1};
                    const f16x2 t = __builtin_convertvector(a2, f16x2);
                    const f32x2 b2 = {a2[0] - (float)t[0], a2[1] - (float)t[1]};
                    hi[i / 2] = __builtin_bit_cast(uint32_t, t);
                    lo[i / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(b2, f16x2));
                }
// by pairs of tiles: the two terms of one would wait for each other
#pragma unroll
                for (int c = g * (G / 16); c < (g + 1) * (G / 16); c += 2) {
                    if (c % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                    const int w = 2 * (c / 4);
                    u32x4 va[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        va[k] = u32x4{centred_pair(cur.v[0][w], (c & 3) + k), centred_pair(cur.v[0][w + 1], (c & 3) + k),
                                      centred_pair(cur.v[1][w], (c & 3) + k), centred_pair(cur.v[1][w + 1], (c & 3) + k)};
                    o[c] = mfma(va[0], hi, o[c]);
                    o[c + 1] = mfma(va[1], hi, o[c + 1]);
                    o[c] = mfma(va[0], lo, o[c]);
                    o[c + 1] = mfma(va[1], lo, o[c + 1]);
                }
            }
            cur = next;
        }
        if (bad_page && lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
    }

    __asm__ volatile("" ::: "memory");  // parameters are read, results may take their place
    // the four waves' parts: out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
    l = row_sum(l);
#pragma unroll
    for (int g = 0; g < NG; ++g) z[g] = row_sum(z[g]);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(512.0f, o[c][i], z[16 * c / G]);
        *(f32x4 *)&lds_o[wave][col][16 * c + 4 * h] = y;
    }
    if (h == 0) {
        lds_ml[wave][0][col] = ref;
        lds_ml[wave][1][col] = l;
    }
    __syncthreads();
    // 16 threads a row
    const int mr = threadIdx.x / 16, part = threadIdx.x % 16;
    const int orow = j.row0 + mr;
    if (orow >= j.rows) return;
    float M = -__builtin_inff(), L = 0.0f, wgt[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds_ml[w][0][mr]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        wgt[w] = M == -__builtin_inff() ? 0.0f : exp2_fast(lds_ml[w][0][mr] - M);
        L += wgt[w] * lds_ml[w][1][mr];
    }
    const int head = j.h * a.R + orow % a.R;
    const int64_t tok = j.q0 + orow / a.R, grow = tok * a.Hq + head;
    const int64_t prow = (int64_t)j.split * a.n_q * a.Hq + grow;
    const float inv = a.ns > 1 ? 1.0f : (L == 0.0f ? 0.0f : 1.0f / L);
    for (int c = part * 4; c < D; c += 64) {
        f32x4 y = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) y += wgt[w] * *(const f32x4 *)&lds_o[w][mr][c];
        y *= inv;
        if (a.ns > 1) {
            *(f32x4 *)(a.part_o + prow * D + c) = y;
        } else {
            store_out<BF>(a, tok, head, c, y);
        }
    }
    if (part == 0) {
        if (a.ns > 1) {
            a.part_ml[prow * 2] = M;
            a.part_ml[prow * 2 + 1] = L;
        } else if (a.lse) {
            a.lse[grow] = lse_of(M, L);
        }
    }
}

// Heads of 256 in groups of 32 have no blocks of 128 rows: those spilled 226
// registers a lane (512 queries over 4096 keys, 4 heads: 254 us, tiles of 16 rows
// 246; 1024 over 8192, 8 heads: 1730 : 1361).
constexpr bool has_prompt(int D, int G) { return D != 256 || G != 32; }

template <int D, int G, bool BF>
hipError_t attend(const Kv4Attn &a, hipStream_t s)
{
    const int64_t blocks = (int64_t)a.ns * a.pool.H * a.B * a.tiles;
    hipError_t e;
    if (!a.prompt) {
        k_kv4_attn<D, G, BF><<<dim3((uint32_t)blocks), dim3(64 * kWaves), 0, s>>>(a);
    } else if constexpr (has_prompt(D, G)) {
        e = launch_rows<D, G, BF, false>(a, (uint32_t)blocks, s);
        if (e != hipSuccess) return e;
    }
    e = hipGetLastError();
    if (e == hipSuccess && a.ns > 1) {
        const dim3 rows((uint32_t)(std::min(a.n_q, (int64_t)a.B * a.max_q) * a.Hq));  // as many as sequences may have
        if (a.ns <= 8)
            k_kv4_join<D, BF, 64><<<rows, dim3(64), 0, s>>>(a);
        else
            k_kv4_join<D, BF, 512><<<rows, dim3(512), 0, s>>>(a);  // 64 splits of 64 rows: 4.7 us; 79 by 256 threads a third longer
        e = hipGetLastError();
    }
    return e;
}

template <int D, int G>
hipError_t attend_dt(const Kv4Attn &a, bool bf16, hipStream_t s)
{
    return bf16 ? attend<D, G, true>(a, s) : attend<D, G, false>(a, s);
}

}  // namespace

// Which kernel, and how many ways a row's keys are split.
//
// Blocks of 128 rows unpack a key once for all of them, but are few and long:
// they are taken where every sequence may fill one, the keys are 2048 or more
// and blocks and thousands of keys together occupy the chip (8 kv heads of
// 128, R = 4, us a call with its join, this kernel : tiles of 16 rows: 2048
// queries over 8192 keys 505 : 662, 2 x 512 over 4096 156 : 193, 8 x 32 over
// 4096 57 : 73, 128 over 16000 101 : 118, 512 over 4096 with 4 heads of 256
// 149 : 196; not for 1 x 64 over 4096 41 : 28, nor 1024 over 1024 55 : 43).
// Split: two blocks a compute unit (2 x up to 512 over up to 4096, fp16, in two
// 155, unsplit 212, in eight 187), 512 keys or more each.
//
// Tiles of 16 rows: a split costs a block's start and its part of the join, so
// 512 keys or fewer are not split (1 x 300 keys 9.2 us, in two 10.9), else it
// gets at least 256 keys while the blocks are fewer than the compute units,
// 512 up to two blocks a unit (D = 256: a unit holds one), 1024 beyond, up to
// eight a unit, which even out unequal sequences (us a call, this rule against
// its neighbours: 1 x 4000 keys 11.7, in 8 14.7, in 64 14.2; 1 x 16000 15.2, in
// 16 18.8, in 64 16.5; 64 x up to 8192 93, unsplit 106, in 8 99; 64 x up to
// 1000 20, in two 27).  Fewer than four blocks a unit are rounded down to as
// many on every unit where that takes no more than a quarter of them (on 8
// heads 1 x 80000, 79 ways 35, 64 ways 32; 1 x 100000, 98 ways 43, 96 ways 37;
// 2 x 40000, 40 ways 33, 32 ways 30).
namespace {

int64_t prompt_splits(const Kv4Pool &p, int64_t blocks, int64_t keys)
{
    const int64_t ns = std::min((p.D == 256 ? 256 : 512) / blocks, (keys + 511) / 512);
    return std::min<int64_t>(std::max<int64_t>(ns, 1), 128);
}

int64_t narrow_splits(const Kv4Pool &p, int64_t blocks, int64_t keys)
{
    const int64_t level[3][2] = {{256, 256}, {p.D == 256 ? 256 : 512, 512}, {2048, 1024}};  // blocks, keys
    int64_t ns = 1;
    if (keys > 512)
        for (int i = 0; i < 3; ++i) ns = std::max(ns, std::min(level[i][0] / blocks, (keys + level[i][1] - 1) / level[i][1]));
    ns = std::min<int64_t>(ns, 128);
    const int64_t even = ns * blocks / 256 * 256 / blocks;
    return ns * blocks < 1024 && even * 4 >= ns * 3 ? even : ns;
}

}  // namespace

Kv4Plan kv4_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window)
{
    Kv4Plan plan;
    // keys that a block of `rows` rows sees at most
    const auto keys_of = [&](int rows) { return window ? std::min(max_keys, window + rows / R + 1) : max_keys; };
    const int64_t wide_tiles = (max_q * R + kRows - 1) / kRows, tiles = (max_q * R + 15) / 16;
    const int64_t wide = std::max<int64_t>(n_seqs * p.H * wide_tiles, 1), narrow = std::max<int64_t>(n_seqs * p.H * tiles, 1);
    const int64_t keys = keys_of(kRows);
    plan.prompt = has_prompt(p.D, p.G) && max_q * R >= kRows && keys >= 2048 && wide * ((keys + 1023) / 1024) >= 256;
    plan.tiles = (int32_t)(plan.prompt ? wide_tiles : tiles);
    plan.ns = (int32_t)(plan.prompt ? prompt_splits(p, wide, keys) : narrow_splits(p, narrow, keys_of(16)));
    // either kernel's splits grow with the keys, so no window takes more than these
    plan.most_ns = (int32_t)std::max(narrow_splits(p, narrow, max_keys), plan.prompt ? prompt_splits(p, wide, max_keys) : 1);
    return plan;
}

hipError_t launch_kv4_attention(const Kv4Attn &a, bool bf16, hipStream_t stream)
{
    switch (a.pool.D * 1000 + a.pool.G) {
    case 64032: return attend_dt<64, 32>(a, bf16, stream);
    case 64064: return attend_dt<64, 64>(a, bf16, stream);
    case 128032: return attend_dt<128, 32>(a, bf16, stream);
    case 128064: return attend_dt<128, 64>(a, bf16, stream);
    case 128128: return attend_dt<128, 128>(a, bf16, stream);
    case 256032: return attend_dt<256, 32>(a, bf16, stream);
    case 256064: return attend_dt<256, 64>(a, bf16, stream);
    default: return attend_dt<256, 128>(a, bf16, stream);
    }
}
