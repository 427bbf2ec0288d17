// The linear layer with 4-bit weights and group scales ("W4") for gfx950:
// tiled weight layout, the product kernel for few token rows, entry points.
//
// Mathematics: y[m][n] = xs[m] * sum_g s[n][g] * sum_{k in g} xq[m][k] * (q[n][k] - z[n][g]).
// The inner sums are exact INT32 products on the INT8 matrix instructions;
// only the outer sum over the groups is fp32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

// --------------------------------------------------------------- tiled layout

// Fragment (tile t of 16 channels, block b of 128 columns) is 1 KiB at
// (t * KB + b) * 1024, KB = ceil(K/128).  Lane L = n + 16 g of a wave owns 16
// bytes of it, those of channel 16 t + n; byte i holds the code of column
// 128 b + c(g, i) in its low nibble and of column 128 b + 64 + c(g, i) in its
// high one.  The low nibbles of a fragment are thus one B operand of the INT8
// products over columns 0..63 of the block, and the high ones one over
// 64..127, each after one mask.  c(g, i) is 16 g + i (v_mfma_i32_16x16x64_i8
// on activations read 16 bytes at a time), or, with 4 scales a block,
// 32 (i / 8) + 8 g + i % 8: each half of 8 bytes is then an operand of
// v_mfma_i32_16x16x32_i8, whose sum stays inside one 32-column group.
// Without zero points the nibbles are q - 8 in two's complement: masked into
// the high half of a byte they are 16 (q - 8), an INT8 operand in one or two
// instructions for four weights, and the factor 16 is taken out of the fp32
// sum (exactly).  With zero points the nibbles are q.
//
// The scales follow the fragments: P = 1, 2 or 4 per channel and block (the
// group size a multiple of 128, of 64 or of 32; larger groups repeat theirs),
// [t][b][n][P] bf16, then the zero points in the same order, a byte each.
constexpr int kBlk = 128;

int per_block(int64_t K, int64_t group) {
    if (group % 128 == 0 || group >= K) return 1;
    return group % 64 == 0 ? 2 : 4;
}

int64_t w4_bytes(int64_t N, int64_t K, int64_t group, bool zeros) {
    const int64_t frags = ((N + 15) / 16) * ((K + kBlk - 1) / kBlk);
    return frags * (1024 + per_block(K, group) * (zeros ? 48 : 32));
}

__host__ __device__ constexpr int frag_column(int P, int g, int i) {
    return P == 4 ? 32 * (i >> 3) + 8 * g + (i & 7) : 16 * g + i;
}

constexpr int kTileThreads = 256;

// One thread per 16-byte piece, then one per (channel, block) of the scales.
__global__ __launch_bounds__(kTileThreads) void w4_tile_kernel(const uint8_t *__restrict__ packed,
                                                               const uint16_t *__restrict__ scales,
                                                               const uint8_t *__restrict__ zeros, int N, int K,
                                                               int64_t group, int G, int P, int64_t frags,
                                                               uint8_t *__restrict__ tiled) {
    const int KB = (K + kBlk - 1) / kBlk;
    uint16_t *sc = reinterpret_cast<uint16_t *>(tiled + frags * 1024);
    uint8_t *zp = tiled + frags * (1024 + 32 * P);
    const int64_t pieces = frags * 64, total = pieces + frags * 16;
    for (int64_t c = (int64_t)blockIdx.x * kTileThreads + threadIdx.x; c < total;
         c += (int64_t)gridDim.x * kTileThreads) {
        const bool piece = c < pieces;
        const int64_t f = piece ? c >> 6 : (c - pieces) >> 4;
        const int l = piece ? (int)(c & 63) : (int)((c - pieces) & 15);
        const int64_t tile = f / KB;
        const int64_t n = tile * 16 + (l & 15);
        const int k0 = (int)(f - tile * KB) * kBlk;
        if (piece) {
            auto code = [&](int k) -> uint32_t {
                if (n >= N || k >= K) return 0u;
                const uint32_t q = (packed[n * (K / 2) + k / 2] >> (4 * (k & 1))) & 15u;
                return zeros ? q : q ^ 8u;
            };
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int k = k0 + frag_column(P, l >> 4, i);
                w[i >> 2] |= (code(k) | (code(k + 64) << 4)) << (8 * (i & 3));
            }
            *reinterpret_cast<uint4 *>(tiled + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int p = 0; p < P; ++p) {
                const int k = k0 + p * (kBlk / P);
                const bool ok = n < N && k < K;
                const int64_t at = ok ? n * G + k / group : 0;
                sc[(f * 16 + l) * P + p] = ok ? scales[at] : (uint16_t)0;
                if (zeros) zp[(f * 16 + l) * P + p] = ok ? zeros[at] : (uint8_t)0;
            }
        }
    }
}

// --------------------------------------------------------------- decode

// INT8 B operand dwords of the low (h = 0) or high (h = 1) nibbles of packed
// dword w.  Without zero points: 16 (q - 8) per byte.  With: q - z, where zrep
// holds z in every byte (the set top bit keeps each byte's difference from
// borrowing out of it; clearing it by exclusive or leaves q - z).
template <bool kZeros>
__device__ __forceinline__ int32_t nibbles(uint32_t w, int h, uint32_t zrep) {
    if constexpr (kZeros) {
        const uint32_t q = (h ? w >> 4 : w) & 0x0F0F0F0Fu;
        return (int32_t)(((q | 0x80808080u) - zrep) ^ 0x80808080u);
    } else {
        return (int32_t)((h ? w : w << 4) & 0xF0F0F0F0u);
    }
}

// --------------------------------------------------------------- product, few rows

// Token rows 16 R at a time against NT tiles of 16 channels, the columns split
// over the waves.  A workgroup's W waves form W / KS teams; a team takes a
// group of NT tiles at a time, its KS waves every KS-th block of 128 columns.
// Both operands go straight from memory to registers in operand order (lane
// L = n + 16 g: B column n; A row n, 16-byte piece g), kDepth blocks ahead;
// nothing passes through LDS but the waves' partial sums, which a team adds in
// wave order.
//
// A row r of a row tile is token 4 (r % 4) + r / 4, so that result register i
// of lane group g belongs to token 4 i + g: with up to 4 tokens only register
// 0 of every result is converted and scaled, with up to 8 two (Q registers).
template <int R, int NT, int Q, int P, bool kZeros, int W>
__global__ __launch_bounds__(W * 64) void w4_rows_kernel(const int8_t *__restrict__ xq, const float *__restrict__ xs,
                                                         const uint8_t *__restrict__ tiled, int M, int K, int N,
                                                         int KS, int rounds, int wgs, void *__restrict__ y, int obf) {
    constexpr int kDepth = 2;
    __shared__ float red[W * NT * R * Q * 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int KB = (K + kBlk - 1) / kBlk, tiles = (N + 15) >> 4;
    const int teams = W / KS, team = wave / KS, part = wave - team * KS;
    const int bm = (int)blockIdx.x / wgs, bc = (int)blockIdx.x - bm * wgs;  // row tile, place among its wgs workgroups
    const int m0 = bm * 16 * R;
    const uint32_t frags = (uint32_t)tiles * (uint32_t)KB;
    const auto rx = make_rsrc(xq, (uint32_t)M * (uint32_t)K);
    const auto rw = make_rsrc(tiled, frags * 1024u);
    const auto rs = make_rsrc(tiled + (int64_t)frags * 1024, frags * (32u * P));
    const auto rz = make_rsrc(tiled + (int64_t)frags * (1024 + 32 * P), kZeros ? frags * (16u * P) : 0u);

    struct Stage {
        uint4 w[NT];
        uint32_t s[NT][P == 4 ? 2 : 1], z[NT];
        uint4 a[R][2];
    };
    const int steps_tile = (KB - part + KS - 1) / KS;  // this wave's blocks of a tile group
    int group = bc * teams + team;        // of the next step to load
    const int stride = wgs * teams;
    uint32_t arow[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int tok = m0 + 16 * r + 4 * (n & 3) + (n >> 2);
        arow[r] = tok < M ? (uint32_t)tok * (uint32_t)K : kOOB;
    }
    auto load = [&](Stage &st, int grp, int step) {
        const int kb = part + KS * step;
        const bool live = step < steps_tile;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (P == 4) {
                    // the columns of byte halves 0..7 and 8..15 of the fragment's lane
                    const int k = kb * kBlk + 64 * h + 8 * g;
                    const uint32_t o0 = live && arow[r] != kOOB && k < K ? arow[r] + (uint32_t)k : kOOB;
                    const uint32_t o1 = live && arow[r] != kOOB && k + 32 < K ? arow[r] + (uint32_t)k + 32u : kOOB;
                    const auto lo = __builtin_amdgcn_raw_buffer_load_b64(rx, o0, 0, 0);
                    const auto hi = __builtin_amdgcn_raw_buffer_load_b64(rx, o1, 0, 0);
                    st.a[r][h] = make_uint4(lo[0], lo[1], hi[0], hi[1]);
                } else {
                    const int k = kb * kBlk + 64 * h + 16 * g;
                    st.a[r][h] = bload16(rx, live && arow[r] != kOOB && k < K ? arow[r] + (uint32_t)k : kOOB);
                }
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int tile = grp * NT + t;
            const uint32_t f = (uint32_t)tile * (uint32_t)KB + (uint32_t)kb;
            const bool ok = live && tile < tiles;
            st.w[t] = bload16(rw, ok ? f * 1024u + 16u * (uint32_t)lane : kOOB);
            const uint32_t so = ok ? (f * 16u + (uint32_t)n) * (2u * P) : kOOB;
            if constexpr (P == 1) {
                st.s[t][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, so, 0, 0);
            } else if constexpr (P == 2) {
                st.s[t][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, so, 0, 0);
            } else {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, so, 0, 0);
                st.s[t][0] = v[0];
                st.s[t][1] = v[1];
            }
            if constexpr (kZeros) {
                const uint32_t zo = ok ? (f * 16u + (uint32_t)n) * (uint32_t)P : kOOB;
                if constexpr (P == 1) st.z[t] = __builtin_amdgcn_raw_buffer_load_b8(rz, zo, 0, 0);
                if constexpr (P == 2) st.z[t] = __builtin_amdgcn_raw_buffer_load_b16(rz, zo, 0, 0);
                if constexpr (P == 4) st.z[t] = __builtin_amdgcn_raw_buffer_load_b32(rz, zo, 0, 0);
            }
        }
    };
    float sum[NT][R][Q];
    auto consume = [&](const Stage &st) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t wv[4] = {st.w[t].x, st.w[t].y, st.w[t].z, st.w[t].w};
            v4i acc[R];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i b;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int p = P == 1 ? 0 : P == 2 ? h : 2 * h + (d >> 1);
                    const uint32_t zrep = kZeros ? ((st.z[t] >> (8 * p)) & 0xFFu) * 0x01010101u : 0u;
                    b[d] = nibbles<kZeros>(wv[d], h, zrep);
                }
                auto add = [&](const v4i &c, int r, uint32_t sbits) {
                    const float s = __uint_as_float(sbits << 16);
#pragma unroll
                    for (int i = 0; i < Q; ++i) sum[t][r][i] = __builtin_fmaf(s, (float)c[i], sum[t][r][i]);
                };
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint4 av = st.a[r][h];
                    const v4i a = {(int)av.x, (int)av.y, (int)av.z, (int)av.w}, zero = {0, 0, 0, 0};
                    if constexpr (P == 4) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const long al = (long)((uint64_t)(uint32_t)a[2 * e] | (uint64_t)(uint32_t)a[2 * e + 1] << 32);
                            const long bl = (long)((uint64_t)(uint32_t)b[2 * e] | (uint64_t)(uint32_t)b[2 * e + 1] << 32);
                            const v4i c = __builtin_amdgcn_mfma_i32_16x16x32_i8(al, bl, zero, 0, 0, 0);
                            add(c, r, e ? st.s[t][h] >> 16 : st.s[t][h]);
                        }
                    } else if constexpr (P == 2) {
                        const v4i c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, zero, 0, 0, 0);
                        add(c, r, h ? st.s[t][0] >> 16 : st.s[t][0]);
                    } else {
                        acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, h ? acc[r] : zero, 0, 0, 0);
                        if (h) add(acc[r], r, st.s[t][0]);
                    }
                }
            }
        }
    };

    Stage ring[kDepth];
    // (group, step) of the next load; every wave of a team loads and consumes
    // in the same order, blocks past its share are predicated off
    int ld_group = group, ld_step = 0;
    const int steps_max = (KB + KS - 1) / KS;  // of any wave, so that barriers line up
    auto load_next = [&](Stage &st) {
        load(st, ld_group, ld_step);
        if (++ld_step == steps_max) {
            ld_step = 0;
            ld_group += stride;
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load_next(ring[d]);

    const float post = kZeros ? 1.0f : 0.0625f;
    auto clear = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < Q; ++i) sum[t][r][i] = 0.0f;
    };
    clear();
    int step = 0;
    const int total = rounds * steps_max;
#pragma unroll 1
    for (int st0 = 0; st0 < total; st0 += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            if (st0 + u >= total) break;  // uniform
            consume(ring[u]);
            load_next(ring[u]);
            if (++step < steps_max) continue;
            // the team's partial sums of this tile group, added in wave order
            step = 0;
            float *mine = red + wave * (NT * R * Q * 64);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < Q; ++i) mine[((t * R + r) * Q + i) * 64 + lane] = sum[t][r][i];
            clear();
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const float *from = red + team * KS * (NT * R * Q * 64);
            for (int o = part * 64 + lane; o < NT * R * Q * 64; o += KS * 64) {
                // o = ((r Q + i) 4 + g') (16 NT) + channel
                const int ch = o % (16 * NT), tk = o / (16 * NT);
                const int gg = tk & 3, ri = tk >> 2, i = ri % Q, r = ri / Q;
                const int m = m0 + 16 * r + 4 * i + gg, c = group * (16 * NT) + ch;
                const float *at = from + (((ch >> 4) * R + r) * Q + i) * 64 + (ch & 15) + 16 * gg;
                float v = 0.0f;
                for (int w = 0; w < KS; ++w) v += at[w * (NT * R * Q * 64)];
                if (m < M && c < N) {
                    v = xs[m] * (v * post);
                    if (obf)
                        static_cast<uint16_t *>(y)[(int64_t)m * N + c] = f32_to_bf16_rne(v);
                    else
                        static_cast<float *>(y)[(int64_t)m * N + c] = v;
                }
            }
            group += stride;
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    }
}

// --------------------------------------------------------------- product, many rows

// Workgroup tile of 16 TR WR token rows x 16 TC (8 / WR) channels on eight
// waves, each with TR x TC results of 16 x 16.  Everything a block of 128
// columns needs is copied to LDS by LDS-DMA, S - 1 blocks ahead: the
// activations, shared by the waves and stored in A operand order (every operand
// read is contiguous, no bank conflicts), and each wave's own fragments,
// scales and zero points.  (With the fragments loaded into registers instead,
// the compiler's waits for them count only the loads it knows and so also wait
// for younger activation copies.)
template <int TR, int TC, int WR, int KP, int S, int P, bool kZeros>
__global__ __launch_bounds__(512, TR * TC <= 16 ? 4 : 2) void w4_gemm_kernel(
    const int8_t *__restrict__ xq, const uint8_t *__restrict__ tiled, int M, int K, int N, int nbm, int nbn,
    const float *__restrict__ xs, void *__restrict__ y, int obf) {
    constexpr int WP = 8 / KP;                     // waves of a column range
    constexpr int BM = 16 * TR * WR, WC = WP / WR, BN = 16 * TC * WC;
    constexpr int NA = BM / 8 / WP;                // activation loads (1 KiB) per wave and block
    constexpr int NL = NA + TC + (kZeros ? 2 : 1);  // all loads per wave and block
    static_assert(BM / 8 % WP == 0, "the waves of a range share its activation loads evenly");
    static_assert(TC * 8 * P <= 64, "a wave's scales of a block are one load of 4 bytes per lane");
    constexpr int kRangeBytes = BM * kBlk, kLds = KP * S * kRangeBytes;
    constexpr int kSumBytes = KP > 1 ? 8 * TR * TC * 1024 : 0;  // partial sums, after the last block
    __shared__ __attribute__((aligned(16))) int8_t abuf[kLds > kSumBytes ? kLds : kSumBytes];
    __shared__ __attribute__((aligned(16))) uint8_t wbuf[S][8][TC * 1024];
    __shared__ __attribute__((aligned(16))) uint8_t sbuf[S][8][256], zbuf[kZeros ? S : 1][8][256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int KB = (K + kBlk - 1) / kBlk, tiles = (N + 15) >> 4;
    int bm, bn;
    if (!gemm_tile(nbm, nbn, bm, bn)) return;  // padding workgroup
    const int part = wave / WP, pw = wave - part * WP;  // column range, wave of it
    const int row0 = bm * BM, wr = pw / WC, tile0 = bn * (BN / 16) + (pw - wr * WC) * TC;
    const int steps = (KB + KP - 1) / KP;

    const uint32_t frags = (uint32_t)tiles * (uint32_t)KB;
    const v4i rx = rsrc_words(xq, (uint32_t)M * (uint32_t)K);
    const v4i rw = rsrc_words(tiled, frags * 1024u);
    const v4i rs = rsrc_words(tiled + (int64_t)frags * 1024, frags * (32u * P));
    const v4i rz = rsrc_words(tiled + (int64_t)frags * (1024 + 32 * P), kZeros ? frags * (16u * P) : 0u);

    // activation load L = pw + WP j: rows 16 (L / 2) .., columns 64 (L % 2) ..
    // of a block, chunk g of row n at 16 lane of KiB L
    uint32_t aoff[NA], atail[NA];
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int L = pw + WP * j, row = row0 + 16 * (L >> 1) + n, col = 64 * (L & 1) + 16 * g;
        aoff[j] = row < M ? (uint32_t)row * (uint32_t)K + (uint32_t)col : kOOB;
        atail[j] = (KB - 1) * kBlk + col < K ? aoff[j] : kOOB;
    }
    // scale load: dword `lane` of the wave's TC tiles of 8 P dwords; zero
    // points: of 4 P dwords.  (A tile past the last one re-reads that one: its
    // channels are not stored.)
    auto first = [&](int t) { return (uint32_t)min(tile0 + t, tiles - 1) * (uint32_t)KB; };
    const uint32_t st = (uint32_t)lane / (8 * P), zt = (uint32_t)lane / (4 * P);
    const uint32_t soff = st < TC ? first(st) * (32u * P) + 4u * (lane % (8 * P)) : kOOB;
    const uint32_t zoff = zt < TC ? first(zt) * (16u * P) + 4u * (lane % (4 * P)) : kOOB;
    uint32_t wfirst[TC];
#pragma unroll
    for (int t = 0; t < TC; ++t) wfirst[t] = __builtin_amdgcn_readfirstlane(first(t) * 1024u);
    const uint32_t alds = S3D8_LDS_OFFSET(&abuf[0]) + (uint32_t)(kRangeBytes * part) + 1024u * (uint32_t)pw;
    const uint32_t wlds = S3D8_LDS_OFFSET(&wbuf[0][wave][0]);
    const uint32_t slds = S3D8_LDS_OFFSET(&sbuf[0][wave][0]), zlds = S3D8_LDS_OFFSET(&zbuf[0][wave][0]);
    // step i of column range `part` is block part + KP i.  Past the last block
    // the activations are zeros and the weights those of the last one, so
    // that every wait counts the same and every range takes as many steps.
    auto issue = [&](int i, int slot) {
        const int kb = part + KP * i;
        const uint32_t kbc = (uint32_t)min(kb, KB - 1);
#pragma unroll
        for (int j = 0; j < NA; ++j)
            load_to_lds16_so(alds + (uint32_t)(KP * kRangeBytes) * slot + (uint32_t)(WP * 1024) * j,
                             kb < KB - 1 ? aoff[j] : kb == KB - 1 ? atail[j] : kOOB, kbc * kBlk, rx);
#pragma unroll
        for (int t = 0; t < TC; ++t)
            load_to_lds16_so(wlds + (8u * TC * 1024u) * slot + 1024u * t, 16u * lane, wfirst[t] + kbc * 1024u, rw);
        load_to_lds4_so(slds + 2048u * slot, soff, kbc * (32u * P), rs);
        if constexpr (kZeros) load_to_lds4_so(zlds + 2048u * slot, zoff, kbc * (16u * P), rz);
    };

    float4 sum[TR][TC];
#pragma unroll
    for (int r = 0; r < TR; ++r)
#pragma unroll
        for (int t = 0; t < TC; ++t) sum[r][t] = make_float4(0, 0, 0, 0);
    typedef int32_t v2i __attribute__((ext_vector_type(2)));
    auto add = [&](float4 &o, const v4i &c, float s) {
        o.x = __builtin_fmaf(s, (float)c[0], o.x);
        o.y = __builtin_fmaf(s, (float)c[1], o.y);
        o.z = __builtin_fmaf(s, (float)c[2], o.z);
        o.w = __builtin_fmaf(s, (float)c[3], o.w);
    };

#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i, i);
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
        // this wave's copies of step i have landed, everyone's after the
        // barrier, which also ends every read of step i - 1's slot
        wait_vmcnt_barrier<(S - 2) * NL>();
        issue(i + S - 1, slot == 0 ? S - 1 : slot - 1);
        v4i b[2][TC];
        float s[TC][P];
#pragma unroll
        for (int t = 0; t < TC; ++t) {
            const uint4 w = *reinterpret_cast<const uint4 *>(&wbuf[slot][wave][1024 * t + 16 * lane]);
            const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
            uint32_t sv[2] = {0, 0}, zv = 0;
            const uint8_t *sp = &sbuf[slot][wave][32 * P * t + 2 * P * n], *zp = &zbuf[kZeros ? slot : 0][wave][16 * P * t + P * n];
            if constexpr (P == 1) sv[0] = *reinterpret_cast<const uint16_t *>(sp);
            if constexpr (P == 2) sv[0] = *reinterpret_cast<const uint32_t *>(sp);
            if constexpr (P == 4) {
                const uint2 v = *reinterpret_cast<const uint2 *>(sp);
                sv[0] = v.x;
                sv[1] = v.y;
            }
            if constexpr (kZeros) {
                if constexpr (P == 1) zv = *zp;
                if constexpr (P == 2) zv = *reinterpret_cast<const uint16_t *>(zp);
                if constexpr (P == 4) zv = *reinterpret_cast<const uint32_t *>(zp);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int p = P == 1 ? 0 : P == 2 ? h : 2 * h + (d >> 1);
                    b[h][t][d] = nibbles<kZeros>(wv[d], h, kZeros ? ((zv >> (8 * p)) & 0xFFu) * 0x01010101u : 0u);
                }
#pragma unroll
            for (int p = 0; p < P; ++p) s[t][p] = __uint_as_float(p & 1 ? sv[p >> 1] & 0xFFFF0000u : sv[p >> 1] << 16);
        }
        // The products in TR P steps of TC results each.  A step reads the
        // next one's activations, issues its own products and scales the
        // previous step's results, so that neither the reads nor the products
        // are waited for.
        const int8_t *at = &abuf[kRangeBytes * (KP * slot + part) + wr * TR * 2048];
        const v4i zero = {0, 0, 0, 0};
        constexpr int kSteps = TR * P;
        auto read_a = [&](int i, v4i (&a)[2]) {
            const int r = i / P, p = i % P;
            if constexpr (P == 4) {
                // columns 32 p + 8 g .. + 7 of the block: half g % 2 of chunk 2 (p % 2) + g / 2
                const v2i v = *reinterpret_cast<const v2i *>(at + 2048 * r + 1024 * (p >> 1) + 512 * (p & 1) +
                                                             256 * (g >> 1) + 16 * n + 8 * (g & 1));
                a[0][0] = v[0];
                a[0][1] = v[1];
            } else {
                a[0] = *reinterpret_cast<const v4i *>(at + 2048 * r + 1024 * p + 16 * lane);
                if constexpr (P == 1) a[1] = *reinterpret_cast<const v4i *>(at + 2048 * r + 1024 + 16 * lane);
            }
        };
        auto two = [](int lo, int hi) { return (long)((uint64_t)(uint32_t)lo | (uint64_t)(uint32_t)hi << 32); };
        v4i a[2][2], c[2][TC];
        read_a(0, a[0]);
#pragma unroll
        for (int i = 0; i <= kSteps; ++i) {
            const int p = i % P, now = i & 1;
            if (i + 1 < kSteps) read_a(i + 1, a[now ^ 1]);
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                if (i < kSteps) {
                    if constexpr (P == 4) {
                        const v4i &bv = b[p >> 1][t];
                        const int e = 2 * (p & 1);
                        c[now][t] = __builtin_amdgcn_mfma_i32_16x16x32_i8(two(a[now][0][0], a[now][0][1]),
                                                                          two(bv[e], bv[e + 1]), zero, 0, 0, 0);
                    } else {
                        c[now][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[now][0], b[p][t], zero, 0, 0, 0);
                        if constexpr (P == 1)
                            c[now][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[now][1], b[1][t], c[now][t], 0, 0, 0);
                    }
                }
                if (i > 0) add(sum[(i - 1) / P][t], c[now ^ 1][t], s[t][(i - 1) % P]);
            }
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // the reads
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                __builtin_amdgcn_sched_group_barrier(0x008, P == 1 ? 2 : 1, 0);  // a product
                __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);               // and the scaling of one
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        slot = slot == S - 1 ? 0 : slot + 1;
    }
    wait_vmcnt<0>();  // loads of blocks past the end
    // the ranges' sums, added in their order; the waves of a range then store
    // TR / KP row tiles each
    constexpr int TO = TR / KP;
    static_assert(TR % KP == 0, "the ranges share the row tiles evenly");
    float4 out[TO][TC];
    if constexpr (KP == 1) {
#pragma unroll
        for (int r = 0; r < TO; ++r)
#pragma unroll
            for (int t = 0; t < TC; ++t) out[r][t] = sum[r][t];
    } else {
        wait_vmcnt_barrier<0>();  // every wave has read its last block
        float4 *red = reinterpret_cast<float4 *>(&abuf[0]);
#pragma unroll
        for (int r = 0; r < TR; ++r)
#pragma unroll
            for (int t = 0; t < TC; ++t) red[((part * WP + pw) * TR * TC + r * TC + t) * 64 + lane] = sum[r][t];
        wait_vmcnt_barrier<0>();
#pragma unroll
        for (int r = 0; r < TO; ++r)
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < KP; ++q) {
                    const float4 u = red[((q * WP + pw) * TR * TC + (part * TO + r) * TC + t) * 64 + lane];
                    v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                }
                out[r][t] = v;
            }
    }

    // result lane (n, g), element i: row 4 g + i of the row tile, channel n.
    // Rows past M lie past the end of the buffer and channels past N get an
    // offset that does: those stores are dropped.
    const int wrow = row0 + 16 * (TR * wr + TO * part), nrows = min(M - wrow, 16 * TO);
    if (nrows <= 0) return;
    const uint32_t size = obf ? 2u : 4u, rowb = size * (uint32_t)N;
    const auto ry = make_rsrc(static_cast<char *>(y) + (int64_t)wrow * N * size, rowb * (uint32_t)nrows);
    const auto rxs = make_rsrc(xs + wrow, 4u * (uint32_t)nrows);
    const float post = kZeros ? 1.0f : 0.0625f;
    uint32_t base[TC];
#pragma unroll
    for (int t = 0; t < TC; ++t) {
        const int ch = 16 * (tile0 + t) + n;
        base[t] = ch < N ? 4u * g * rowb + size * (uint32_t)ch : kOOB;
    }
#pragma unroll
    for (int r = 0; r < TO; ++r) {
        const uint4 sx = bload16(rxs, 64u * r + 16u * g);
        const float sxv[4] = {__uint_as_float(sx.x), __uint_as_float(sx.y), __uint_as_float(sx.z), __uint_as_float(sx.w)};
#pragma unroll
        for (int t = 0; t < TC; ++t) {
            const float v[4] = {out[r][t].x, out[r][t].y, out[r][t].z, out[r][t].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t off = base[t] + (uint32_t)(16 * r + i) * rowb;
                const float o = sxv[i] * (v[i] * post);
                if (obf)
                    __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_rne(o), ry, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o), ry, off, 0, 0);
            }
        }
    }
}

// --------------------------------------------------------------- launches

struct W4Args {
    const int8_t *xq;
    const float *xs;
    const uint8_t *tiled;
    int M, K, N;
    void *y;
    int obf;
};

template <int R, int NT, int Q, int W>
void launch_rows(const W4Args &a, int P, bool zeros, int cus, hipStream_t stream) {
    const int KB = (a.K + kBlk - 1) / kBlk, groups = ((a.N + 15) / 16 + NT - 1) / NT;
    // as many waves on one group's columns as it has blocks, until the groups
    // fill the waves of every CU
    int KS = W;
    while (KS > 1 && (KS / 2 >= KB || (int64_t)groups * KS > (int64_t)cus * W * 2)) KS /= 2;
    const int teams = W / KS;
    const int wgs = std::min((groups + teams - 1) / teams, cus);
    const int rounds = (groups + wgs * teams - 1) / (wgs * teams);
    typedef void (*Fn)(const int8_t *, const float *, const uint8_t *, int, int, int, int, int, int, void *, int);
    static const Fn fns[3][2] = {
        {w4_rows_kernel<R, NT, Q, 1, false, W>, w4_rows_kernel<R, NT, Q, 1, true, W>},
        {w4_rows_kernel<R, NT, Q, 2, false, W>, w4_rows_kernel<R, NT, Q, 2, true, W>},
        {w4_rows_kernel<R, NT, Q, 4, false, W>, w4_rows_kernel<R, NT, Q, 4, true, W>},
    };
    hipLaunchKernelGGL(fns[P == 4 ? 2 : P - 1][zeros], dim3(wgs * ((a.M + 16 * R - 1) / (16 * R))), dim3(W * 64), 0,
                       stream, a.xq, a.xs, a.tiled, a.M, a.K, a.N, KS, rounds, wgs, a.y, a.obf);
}

// Token rows of one call: keeps every launch under 2^32 threads.
constexpr int64_t kMaxRows = 1 << 19;

// Workgroup tiles of the GEMM: rows and channels, column ranges (waves split
// between them), and the time of a step of `ranges` blocks and of everything
// else, in ns, from K = 4096 with one workgroup on a CU (a second one beside
// it gains little: a workgroup keeps its SIMDs' issue busy).
struct GemmTile {
    int rows, channels, ranges, step_ns, fixed_ns;
};
constexpr GemmTile kGemmTiles[] = {
    {128, 256, 1, 1500, 3000}, {64, 256, 1, 920, 3000}, {64, 128, 2, 950, 3000},
    {64, 64, 4, 1050, 3000},   {32, 128, 2, 620, 3000}, {64, 32, 4, 650, 3000},
};

// The tile with the least estimated time: rounds of workgroups on the CUs
// times a workgroup's time.
int gemm_tile_choice(int64_t M, int64_t K, int64_t N, int cus) {
    const int64_t KB = (K + kBlk - 1) / kBlk;
    int best = 0;
    int64_t least = 0;
    for (int i = 0; i < (int)(sizeof(kGemmTiles) / sizeof(kGemmTiles[0])); ++i) {
        const GemmTile &t = kGemmTiles[i];
        const int64_t wgs = ((M + t.rows - 1) / t.rows) * ((N + t.channels - 1) / t.channels);
        const int64_t ns = ((wgs + cus - 1) / cus) * ((KB + t.ranges - 1) / t.ranges * t.step_ns + t.fixed_ns);
        if (i == 0 || ns < least) {
            least = ns;
            best = i;
        }
    }
    return best;
}

// a wave's rows of output stay under 2^31 bytes (32-bit store offsets)
constexpr int64_t kGemmMaxN = (int64_t(1) << 31) / (4 * 128) - 1;

template <int TR, int TC, int WR, int KP, int S>
void launch_gemm(const W4Args &a, int P, bool zeros, hipStream_t stream) {
    constexpr int BM = 16 * TR * WR, BN = 16 * TC * (8 / KP / WR);
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    typedef void (*Fn)(const int8_t *, const uint8_t *, int, int, int, int, int, const float *, void *, int);
    static const Fn fns[3][2] = {
        {w4_gemm_kernel<TR, TC, WR, KP, S, 1, false>, w4_gemm_kernel<TR, TC, WR, KP, S, 1, true>},
        {w4_gemm_kernel<TR, TC, WR, KP, S, 2, false>, w4_gemm_kernel<TR, TC, WR, KP, S, 2, true>},
        {w4_gemm_kernel<TR, TC, WR, KP, S, 4, false>, w4_gemm_kernel<TR, TC, WR, KP, S, 4, true>},
    };
    hipLaunchKernelGGL(fns[P == 4 ? 2 : P - 1][zeros], dim3((nbm * nbn + kXcds - 1) / kXcds * kXcds), dim3(512), 0,
                       stream, a.xq, a.tiled, a.M, a.K, a.N, nbm, nbn, a.xs, a.y, a.obf);
}

int check_w4(int64_t M, int64_t K, int64_t N, int64_t group, bool zeros) {
    if (M <= 0 || K <= 0 || N <= 0 || group <= 0)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes and group must be positive");
    if (K % 16 != 0) return s3d8::fail(S3D8_ERR_SHAPE, "K must be a multiple of 16");
    if (group % 32 != 0) return s3d8::fail(S3D8_ERR_SHAPE, "group must be a multiple of 32");
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (M > kMaxRows || K > lim - kBlk || N > lim - 64 || M > lim / K || M > lim / N || (N + 15) / 16 > lim / (K + kBlk) ||
        w4_bytes(N, K, group, zeros) > lim)
        return s3d8::fail(S3D8_ERR_SHAPE, "tensor too large (more than 2^31 elements or tiled bytes, or 524288 rows)");
    return S3D8_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_linear(const int8_t *xq, const float *xs, int64_t M, int64_t K, int64_t N, const uint8_t *tiled,
                 int64_t tiled_bytes, int64_t group, int32_t has_zeros, const void *y, int32_t out_type) {
    if (!xq || !xs || !tiled || !y) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    if (out_type != S3D8_OUT_F32 && out_type != S3D8_OUT_BF16)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown output type");
    if (has_zeros != 0 && has_zeros != 1) return s3d8::fail(S3D8_ERR_INVALID_ARG, "has_zeros must be 0 or 1");
    int rc = check_w4(M, K, N, group, has_zeros != 0);
    if (rc) return rc;
    if (tiled_bytes != w4_bytes(N, K, group, has_zeros != 0))
        return s3d8::fail(S3D8_ERR_INVALID_ARG,
                          "tiled_bytes is not s3d8_w4_tiled_bytes(N, K, group, has_zeros): pass the matrix as "
                          "s3d8_w4_tile laid it out for these arguments");
    if (!aligned16(xq) || !aligned16(tiled))
        return s3d8::fail(S3D8_ERR_ALIGN, "xq and the tiled weights must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(xs) & 3u || reinterpret_cast<uintptr_t>(y) & (out_type == S3D8_OUT_F32 ? 3u : 1u))
        return s3d8::fail(S3D8_ERR_ALIGN, "xs and y must be aligned to their elements");
    return S3D8_OK;
}

int launch_linear(const int8_t *xq, const float *xs, int64_t M, int64_t K, int64_t N, const uint8_t *tiled,
                  int64_t group, bool zeros, void *y, int32_t out_type, int cus, hipStream_t stream) {
    const W4Args a{xq, xs, tiled, (int)M, (int)K, (int)N, y, out_type == S3D8_OUT_BF16};
    const int P = per_block(K, group);
    if (M <= 4)
        launch_rows<1, 1, 1, 16>(a, P, zeros, cus, stream);
    else if (M <= 8)
        launch_rows<1, 2, 2, 16>(a, P, zeros, cus, stream);
    else if (M <= 16)
        launch_rows<1, 2, 4, 16>(a, P, zeros, cus, stream);
    else if (N > kGemmMaxN)
        launch_rows<2, 2, 4, 8>(a, P, zeros, cus, stream);
    else
        switch (gemm_tile_choice(M, K, N, cus)) {
            case 0: launch_gemm<8, 2, 1, 1, 2>(a, P, zeros, stream); break;
            case 1: launch_gemm<4, 2, 1, 1, 3>(a, P, zeros, stream); break;
            case 2: launch_gemm<4, 2, 1, 2, 3>(a, P, zeros, stream); break;
            case 3: launch_gemm<4, 2, 1, 4, 3>(a, P, zeros, stream); break;
            case 4: launch_gemm<2, 2, 1, 2, 3>(a, P, zeros, stream); break;
            default: launch_gemm<4, 1, 1, 4, 3>(a, P, zeros, stream); break;
        }
    return s3d8::launch_status();
}

}  // namespace

extern "C" {

int64_t s3d8_w4_tiled_bytes(int64_t N, int64_t K, int64_t group, int32_t has_zeros) {
    if (N <= 0 || K <= 0 || group <= 0 || group % 32 != 0) return -1;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (N > lim || K > lim || (N + 15) / 16 > (int64_t(1) << 50) / (K + kBlk)) return -1;
    return w4_bytes(N, K, group, has_zeros != 0);
}

int32_t s3d8_w4_tile(const uint8_t *packed, const uint16_t *scales_bf16, const uint8_t *zeros, int64_t N, int64_t K,
                     int64_t group, uint8_t *tiled, void *stream) {
    if (!packed || !scales_bf16 || !tiled) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    int rc = check_w4(1, K, N, group, zeros != nullptr);
    if (rc) return rc;
    if (!aligned16(tiled)) return s3d8::fail(S3D8_ERR_ALIGN, "tiled must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(scales_bf16) & 1u)
        return s3d8::fail(S3D8_ERR_ALIGN, "scales_bf16 must be 2-byte aligned");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    const int64_t frags = ((N + 15) / 16) * ((K + kBlk - 1) / kBlk);
    const int64_t blocks = std::min<int64_t>((frags * 80 + kTileThreads - 1) / kTileThreads, (int64_t)cus * 8);
    hipLaunchKernelGGL(w4_tile_kernel, dim3((unsigned)blocks), dim3(kTileThreads), 0, (hipStream_t)stream, packed,
                       scales_bf16, zeros, (int)N, (int)K, group, (int)((K - 1) / group + 1), per_block(K, group),
                       frags, tiled);
    return s3d8::launch_status();
}

int32_t s3d8_w4_linear(const int8_t *xq, const float *xs, int64_t M, int64_t K, int64_t N, const uint8_t *tiled,
                       int64_t tiled_bytes, int64_t group, int32_t has_zeros, void *y, int32_t out_type,
                       void *stream) {
    int rc = check_linear(xq, xs, M, K, N, tiled, tiled_bytes, group, has_zeros, y, out_type);
    if (rc) return rc;
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    return launch_linear(xq, xs, M, K, N, tiled, group, has_zeros != 0, y, out_type, cus, (hipStream_t)stream);
}

int32_t s3d8_w4_forward(const float *x, int64_t M, int64_t K, int64_t N, const uint8_t *tiled, int64_t tiled_bytes,
                        int64_t group, int32_t has_zeros, void *y, int32_t out_type, int8_t *xq, float *xs,
                        void *stream) {
    int rc = check_linear(xq, xs, M, K, N, tiled, tiled_bytes, group, has_zeros, y, out_type);
    if (rc) return rc;
    rc = s3d8_quant_act(x, M, K, xq, xs, stream);
    if (rc) return rc;
    return s3d8_w4_linear(xq, xs, M, K, N, tiled, tiled_bytes, group, has_zeros, y, out_type, stream);
}

}  // extern "C"
