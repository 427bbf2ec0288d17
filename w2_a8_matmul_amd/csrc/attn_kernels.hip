// Attention of query tokens to an encoder's states, for gfx950.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kKeys = 64;       // keys in a block
constexpr int kRows = 32;       // query rows of a wave
constexpr int kMaxSplits = 64;
constexpr int kListed = 1024;   // most blocks of a split among which those that a tile sees are listed
// The maximum that is taken off the scores is only raised when a score is past it by this power
// of 2: p up to 2^8 is as exact in bf16 and fp32 as p up to 1, and most blocks scale nothing.
constexpr float kSlack = 8.0f;

// What the kernels read: a pair is a sequence and a key head, whose R = T * G rows are
// its T query tokens (of all sequences, where they share their states) times the G query
// heads that read this key head, head fastest.
struct Attn {
    const uint16_t *q, *k, *v;
    const int32_t *lens;
    const uint64_t *words;  // [mask sequences][blocks][mask rows] bits of 64 keys, or NULL
    uint16_t *o;
    float *part;            // [splits][pairs][R][D] sums, then [splits][pairs][R] maximum and sum of p
    int64_t q_seq, q_row, q_head, k_seq, k_row, k_head, v_seq, v_row, v_head;
    int64_t word_seq, word_block, word_row;
    int Lq, Lk, G, Hk, D, R, pairs, tiles, splits, shared;
    float scale;            // times log2(e)
};

// Chunk (16 bytes, 8 entries) c of row r of a tile lies at chunk place(c, r) of the row's
// CPR chunks in LDS, so that the sixteen rows that a wide read takes a column from lie in
// different banks (keys), and the four rows that a transposed read takes four
// chunks from (values).
template <int CPR>
__device__ __forceinline__ int key_place(int c, int r) {
    return CPR == 16 ? c ^ (r & 15) : CPR == 8 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3);
}
template <int CPR>
__device__ __forceinline__ int value_place(int c, int r) {
    return CPR == 16 ? c ^ ((r & 3) << 2) : CPR == 8 ? c ^ (((r >> 1) & 1) << 2) : c;
}

// The larger of a lane's value and that of the lane 32 further.
__device__ __forceinline__ float halves_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// sum_j p_j v_j of one row over the keys from `begin` to `end` that it sees: entries
// `lane` and `lane` + 64.
__device__ __forceinline__ void visible_sum(const Attn &a, int64_t q_at, const uint16_t *kp, const uint16_t *vp, int64_t word_at,
                                         float most, int begin, int end, float (&e)[2]) {
    const int lane = threadIdx.x & 63;
    const uint64_t *words = a.words + word_at;
    float q[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) q[n] = lane + 64 * n < a.D ? bf16_to_f32(a.q[q_at + lane + 64 * n]) : 0.0f;
    for (int key = begin; key < end; ++key) {
        if (!(words[(key / kKeys) * a.word_block] >> (key % kKeys) & 1)) continue;
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
            if (lane + 64 * n < a.D) s = __builtin_fmaf(q[n], bf16_to_f32(kp[key * a.k_row + lane + 64 * n]), s);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
        const float p = (float)(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s, a.scale, -most));
#pragma unroll
        for (int n = 0; n < 2; ++n)
            if (lane + 64 * n < a.D) e[n] = __builtin_fmaf(p, bf16_to_f32(vp[key * a.v_row + lane + 64 * n]), e[n]);
    }
}

// A workgroup of kR x kK waves: kR over rows, RT tiles of 32 rows each; kK over keys, each on every
// kK-th block of the split's keys with tiles in LDS of its own, joined at the end.
template <int NK, int ND, int RT, int kR, int kK>
__global__ __launch_bounds__(64 * kR * kK, RT == 1 ? 2 : 1) void attn_kernel(const Attn a) {
    constexpr int Dp = 32 * ND;         // entries of a row in LDS
    constexpr int CPR = Dp / 8;
    constexpr int kTile = kKeys * CPR;  // chunks
    static_assert(16 * NK <= Dp && CPR % kR == 0, "");
    __shared__ __attribute__((aligned(1024))) uint4 tiles[kK][2][2][kTile];
    __shared__ uint64_t seen[kListed / 64];
    __shared__ uint16_t list[kListed];

    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), wr = wave % kR, wk = wave / kR;
    const int pair = (int)blockIdx.x % a.pairs, rest = (int)blockIdx.x / a.pairs;
    const int tile = rest % a.tiles, split = rest / a.tiles;
    const int seq = pair / a.Hk, head = pair % a.Hk;

    int len = a.lens ? global(a.lens)[a.shared ? 0 : seq] : a.Lk;
    len = max(0, min(len, a.Lk));
    const int blocks = (len + kKeys - 1) / kKeys;
    const int begin = (int)((int64_t)blocks * split / a.splits), end = (int)((int64_t)blocks * (split + 1) / a.splits);

    // this lane's rows (past the last: the last again, not stored)
    struct Row {
        int row, b, i, head;
    };
    auto row_of = [&](int rt) {
        const int row = ((tile * kR + wr) * RT + rt) * kRows + col;
        const int rr = min(row, a.R - 1), t = rr / a.G;
        return Row{row, a.shared ? t / a.Lq : seq, a.shared ? t % a.Lq : t, head * a.G + rr % a.G};
    };
    bf8 qf[RT][NK];
    int64_t q_at[RT], word_at[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const Row r = row_of(rt);
        q_at[rt] = r.b * a.q_seq + r.i * a.q_row + r.head * a.q_head;
        word_at[rt] = r.b * a.word_seq + r.i * a.word_row;
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            v4u u = {0, 0, 0, 0};
            if (16 * s + 8 * h < a.D) u = *global(reinterpret_cast<const v4u *>(a.q + q_at[rt] + 16 * s + 8 * h));
            qf[rt][s] = __builtin_bit_cast(bf8, u);
        }
    }

    // the lane's part of each copy of a tile into LDS
    constexpr int kCopies = CPR / kR;
    uint32_t koff[kCopies], voff[kCopies];
#pragma unroll
    for (int n = 0; n < kCopies; ++n) {
        const int c = (wr + n * kR) * 64 + lane, r = c / CPR, p = c % CPR;
        const int kc = key_place<CPR>(p, r), vc = value_place<CPR>(p, r);  // (its own inverse)
        koff[n] = 8 * kc < a.D ? (uint32_t)r * (uint32_t)a.k_row * 2 + kc * 16 : kOOB;
        voff[n] = 8 * vc < a.D ? (uint32_t)r * (uint32_t)a.v_row * 2 + vc * 16 : kOOB;
    }
    const uint16_t *kp = a.k + seq * a.k_seq + head * a.k_head, *vp = a.v + seq * a.v_seq + head * a.v_head;
    // (no block: a buffer of no bytes, zeros)
    auto copy = [&](const uint16_t *p, int64_t stride, int block, const uint4 *to, const uint32_t (&off)[kCopies]) {
        const int rows = min(kKeys, len - block * kKeys) - 1;
        const v4i r = rsrc_words(p + (int64_t)block * kKeys * stride, block < end ? (uint32_t)(rows * stride + a.D) * 2 : 0);
#pragma unroll
        for (int n = 0; n < kCopies; ++n) load_to_lds16_so(S3D8_LDS_OFFSET(to + (wr + n * kR) * 64), off[n], 0, r);
    };
    auto copy_keys = [&](int block, int buf) { copy(kp, a.k_row, block, tiles[wk][0][buf], koff); };
    auto copy_values = [&](int block, int buf) { copy(vp, a.v_row, block, tiles[wk][1][buf], voff); };

    // With a mask, the blocks that any row of the tile sees, by the words of the tile's tokens: a lane a
    // block, a wave every kR kK-th token.
    int count = end - begin;
    const bool sparse = a.words && count <= kListed;
    if (sparse) {
        for (int n = threadIdx.x; n < kListed / 64; n += 64 * kR * kK) seen[n] = 0;
        __syncthreads();
        const int r0 = tile * kR * RT * kRows, t0 = r0 / a.G, t1 = min(r0 + kR * RT * kRows - 1, a.R - 1) / a.G;
        for (int n = 0; n < count; n += 64) {
            const int block = min(begin + n + lane, end - 1);
            uint64_t any = 0;
#pragma unroll 4
            for (int t = t0 + wave; t <= t1; t += kR * kK) {
                const int b = a.shared ? t / a.Lq : seq, i = a.shared ? t % a.Lq : t;
                any |= global(a.words)[b * a.word_seq + i * a.word_row + block * a.word_block];
            }
            const uint64_t bits = __ballot(any != 0 && n + lane < count);
            if (lane == 0) atomicOr((unsigned long long *)&seen[n / 64], (unsigned long long)bits);
        }
        __syncthreads();
        int at = 0;
        for (int n = 0; n < count; n += 64) {
            const uint64_t bits = seen[n / 64];
            if (wave == 0 && bits >> lane & 1)
                list[at + __builtin_amdgcn_mbcnt_hi((uint32_t)(bits >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)bits, 0))] =
                    (uint16_t)(n + lane);
            at += __builtin_popcountll(bits);
        }
        __syncthreads();
        count = __builtin_amdgcn_readfirstlane(at);
    }
    // the n-th block of this wave's keys, or one past the split's
    auto block_at = [&](int n) {
        n = n * kK + wk;
        if (n >= count) return end;
        return begin + (sparse ? __builtin_amdgcn_readfirstlane((int)list[n]) : n);
    };

    f16v acc[RT][ND];
    float most[RT], sum[RT];  // of scaled scores, in powers of 2; this lane's part of the sum
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        most[rt] = -FLT_MAX;
        sum[rt] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[rt][d][r] = 0.0f;
    }

    // a score operand (32 keys, 16 entries) and a value operand (32 entries, 16 keys; transposed by the
    // read: entry by lane, four keys in a row) of a block
    auto key_operand = [&](int buf, int i) {
        const int n = i / 2, r = i % 2 * 32 + col;
        return *reinterpret_cast<const bf8 *>(reinterpret_cast<const char *>(tiles[wk][0][buf]) +
                                              (r * CPR + key_place<CPR>(2 * n + h, r)) * 16);
    };
    auto value_operand = [&](int buf, int i) {
        const int n = i / ND, d = i % ND;
        struct Two {
            s4 x[2];
        } two;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 16 * n + 8 * j + 4 * h + ((lane & 15) >> 2);
            const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            two.x[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s4 *)(reinterpret_cast<const char *>(tiles[wk][1][buf]) +
                                                         (r * CPR + value_place<CPR>(c, r)) * 16 + 8 * (lane & 1)));
        }
        return __builtin_bit_cast(bf8, two);
    };
    struct Words {
        uint64_t w[RT];
    };
    auto load_words = [&](int block) {
        Words u;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            u.w[rt] = a.words && block < end ? global(a.words)[word_at[rt] + block * a.word_block] : ~0ull;
        return u;
    };
    auto inside = [&](int block) {  // the bits of the keys that exist
        const int n = block < end ? len - block * kKeys : 0;
        return n < kKeys ? (1ull << max(n, 0)) - 1 : ~0ull;
    };
    auto most_of = [&](const f16v(&s)[2]) {
        float m = s[0][0];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) m = fmaxf(m, s[kt][r]);
        return m;
    };

    // Scores are transposed: key by register, row by lane.  Block n is weighed and added while the
    // scores of the next block are computed: their products run beside the exponentials, and the
    // largest of them is found beside the products with the values.
    const int steps = (count + kK - 1) / kK;
    if (steps > 0) {
        int block = block_at(0), next = block_at(1);
        Words words = load_words(block), next_words = load_words(next);
        copy_keys(block, 0);
        copy_values(block, 0);
        wait_vmcnt_barrier<0>();
        copy_keys(next, 1);
        f16v s[RT][2], t[RT][2];
        float m[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[rt][0][r] = s[rt][1][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * NK; ++i) {
            const bf8 kf = key_operand(0, i);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                s[rt][i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[rt][i / 2], s[rt][i % 2], 0, 0, 0);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) m[rt] = most_of(s[rt]);

        auto step = [&](int n, int buf, f16v(&s)[RT][2], f16v(&t)[RT][2]) {
            const int later = block_at(n + 2);
            wait_vmcnt_barrier<0>();
            const uint64_t here = inside(block);
            const Words now = words;
            words = next_words;
            next_words = load_words(later);
            copy_keys(later, buf);
            copy_values(next, buf ^ 1);
            block = next;
            next = later;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint64_t word = now.w[rt] & here;
                if (__ballot(word != ~0ull)) {
                    const uint64_t mine = word >> (4 * h);
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const uint32_t bits = (uint32_t)(mine >> (32 * kt));
                            s[rt][kt][r] = bits >> (8 * (r / 4) + r % 4) & 1 ? s[rt][kt][r] : -INFINITY;
                        }
                    m[rt] = most_of(s[rt]);
                }
                m[rt] = halves_max(m[rt]) * a.scale;
                if (__ballot(m[rt] > most[rt] + kSlack)) {
                    const float top = fmaxf(most[rt], m[rt]);
                    const float f = __builtin_amdgcn_exp2f(most[rt] - top);
                    most[rt] = top;
                    sum[rt] *= f;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[rt][d][r] *= f;
                }
            }
            constexpr int kAhead = 4;  // operands in flight
            bf8 operand[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) operand[i] = key_operand(buf ^ 1, i);
            uint32_t pf[RT][16];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int r = 0; r < 16; ++r) t[rt][0][r] = t[rt][1][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * NK; ++i) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    __builtin_amdgcn_sched_barrier(0);
                    t[rt][i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand[i % kAhead], qf[rt][i / 2], t[rt][i % 2], 0, 0, 0);
                    if (rt == RT - 1)
                        operand[i % kAhead] = i + kAhead < 2 * NK ? key_operand(buf ^ 1, i + kAhead)
                                                                  : value_operand(buf, i + kAhead - 2 * NK);
#pragma unroll
                    for (int e = i * 16 / (2 * NK); e < (i + 1) * 16 / (2 * NK); ++e) {
                        bf2 two;
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            two[x] = (__bf16)__builtin_amdgcn_exp2f(
                                __builtin_fmaf(s[rt][e / 8][2 * (e % 8) + x], a.scale, -most[rt]));
                        sum[rt] = __builtin_amdgcn_fdot2_f32_bf16(two, bf2{(__bf16)1.0f, (__bf16)1.0f}, sum[rt], false);
                        pf[rt][e] = __builtin_bit_cast(uint32_t, two);
                    }
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) m[rt] = t[rt][0][0];
#pragma unroll
            for (int i = 0; i < 4 * ND; ++i) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    __builtin_amdgcn_sched_barrier(0);
                    const uint4 p = make_uint4(pf[rt][i / ND * 4], pf[rt][i / ND * 4 + 1], pf[rt][i / ND * 4 + 2], pf[rt][i / ND * 4 + 3]);
                    acc[rt][i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand[(i + 2 * NK) % kAhead],
                                                                              __builtin_bit_cast(bf8, p), acc[rt][i % ND], 0, 0, 0);
                    if (rt == RT - 1 && i + kAhead < 4 * ND) operand[(i + 2 * NK) % kAhead] = value_operand(buf, i + kAhead);
#pragma unroll
                    for (int e = i * 32 / (4 * ND); e < (i + 1) * 32 / (4 * ND); ++e) m[rt] = fmaxf(m[rt], t[rt][e / 16][e % 16]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int n = 0;;) {
            step(n, 0, s, t);
            if (++n >= steps) break;
            step(n, 1, t, s);
            if (++n >= steps) break;
        }
        wait_vmcnt_barrier<0>();  // the last steps' copies have landed before LDS is used again or let go
    }
    if (a.words) {
        // A hidden key has p = 0, but the product with an infinite or NaN value of it is NaN. Rows that
        // are not finite are summed again, one by one, over what they see.
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float z = 0.0f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) z = __builtin_fmaf(acc[rt][d][r], 0.0f, z);
            uint64_t bad = __ballot(z != z);
            bad = (bad | bad >> 32) & 0xFFFFFFFFull;
            while (bad) {
                const int lost = __builtin_ctzll(bad);
                bad &= bad - 1;
                float e[2] = {0.0f, 0.0f};
                for (int n = 0, block; (block = block_at(n)) < end; ++n)
                    visible_sum(a, __shfl((long long)q_at[rt], lost), kp, vp, __shfl((long long)word_at[rt], lost),
                                __shfl(most[rt], lost), block * kKeys, min((block + 1) * kKeys, len), e);
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float x = __shfl(e[d / 2], (32 * d + 8 * (r / 4) + 4 * h + r % 4) & 63);
                        if (col == lost) acc[rt][d][r] = x;
                    }
            }
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sum[rt] += __shfl_xor(sum[rt], 32);

    if constexpr (kK > 1) {
        // the waves over keys joined, one after the other, through the tiles' LDS
        float4 *room = reinterpret_cast<float4 *>(tiles) + wr * (64 * (4 * ND * RT + 1));
        static_assert(kR * 64 * (4 * ND * RT + 1) * 16 <= (int)sizeof(tiles), "");
        for (int g = 1; g < kK; ++g) {
            __syncthreads();
            if (wk == g) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            room[((rt * ND + d) * 4 + q) * 64 + lane] = make_float4(
                                acc[rt][d][4 * q], acc[rt][d][4 * q + 1], acc[rt][d][4 * q + 2], acc[rt][d][4 * q + 3]);
                room[RT * ND * 4 * 64 + lane] = make_float4(most[0], sum[0], most[RT - 1], sum[RT - 1]);
            }
            __syncthreads();
            if (wk == 0) {
                const float4 ms = room[RT * ND * 4 * 64 + lane];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float om = rt ? ms.z : ms.x, os = rt ? ms.w : ms.y, top = fmaxf(most[rt], om);
                    const float f = __builtin_amdgcn_exp2f(most[rt] - top), o = __builtin_amdgcn_exp2f(om - top);
                    most[rt] = top;
                    sum[rt] = __builtin_fmaf(f, sum[rt], o * os);
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 x = room[((rt * ND + d) * 4 + q) * 64 + lane];
                            acc[rt][d][4 * q] = __builtin_fmaf(f, acc[rt][d][4 * q], o * x.x);
                            acc[rt][d][4 * q + 1] = __builtin_fmaf(f, acc[rt][d][4 * q + 1], o * x.y);
                            acc[rt][d][4 * q + 2] = __builtin_fmaf(f, acc[rt][d][4 * q + 2], o * x.z);
                            acc[rt][d][4 * q + 3] = __builtin_fmaf(f, acc[rt][d][4 * q + 3], o * x.w);
                        }
                }
            }
        }
        if (wk) return;
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const Row u = row_of(rt);
        if (u.row >= a.R) continue;
        if (a.splits > 1) {
            const int64_t at = ((int64_t)split * a.pairs + pair) * a.R + u.row;
            const auto p = global(a.part) + at * a.D;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int e = 32 * d + 2 * r + 4 * h;
                    const v4f x = {acc[rt][d][r], acc[rt][d][r + 1], acc[rt][d][r + 2], acc[rt][d][r + 3]};
                    if (e < a.D) *(__attribute__((address_space(1))) v4f *)(p + e) = x;
                }
            if (h == 0) {
                const auto ms = global(a.part) + (int64_t)a.splits * a.pairs * a.R * a.D + 2 * at;
                ms[0] = most[rt];
                ms[1] = sum[rt];
            }
            continue;
        }
        const float f = sum[rt] == 0.0f ? 0.0f : 1.0f / sum[rt];
        const auto o = global(a.o) + (((int64_t)u.b * a.Lq + u.i) * a.Hk * a.G + u.head) * a.D;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
                const int e = 32 * d + 2 * r + 4 * h;
                const bf4 x = {(__bf16)(acc[rt][d][r] * f), (__bf16)(acc[rt][d][r + 1] * f), (__bf16)(acc[rt][d][r + 2] * f),
                               (__bf16)(acc[rt][d][r + 3] * f)};
                if (e < a.D) *(__attribute__((address_space(1))) bf4 *)(o + e) = x;
            }
    }
}

// Partial sums of the splits joined: 4 entries of a row a thread, kLanes threads of a
// row's entries sharing its splits, so that a row's loads are all on their way at once (one
// thread for all of them: 10 us instead of 3 for 32 rows of 26 splits).
struct Partial {
    float most, sum;
    float4 x;
    __device__ __forceinline__ void join(float m, float n, float4 y) {
        const float top = fmaxf(most, m), f = __builtin_amdgcn_exp2f(most - top), g = __builtin_amdgcn_exp2f(m - top);
        most = top;
        sum = __builtin_fmaf(f, sum, g * n);
        x.x = __builtin_fmaf(f, x.x, g * y.x);
        x.y = __builtin_fmaf(f, x.y, g * y.y);
        x.z = __builtin_fmaf(f, x.z, g * y.z);
        x.w = __builtin_fmaf(f, x.w, g * y.w);
    }
};
template <int kLanes>
__global__ __launch_bounds__(256) void attn_join_kernel(const Attn a) {
    constexpr int kRowsHere = 8 / kLanes, kAtOnce = 4;
    __shared__ Partial parts[256];
    const int e = (threadIdx.x & 31) * 4, lane = (threadIdx.x >> 5) % kLanes, here = (threadIdx.x >> 5) / kLanes;
    const int64_t rows = (int64_t)a.pairs * a.R, at = (int64_t)blockIdx.x * kRowsHere + here;
    const bool in = at < rows && e < a.D;
    const float *ms = a.part + a.splits * rows * a.D;
    Partial p{-FLT_MAX, 0.0f, make_float4(0, 0, 0, 0)};
    if (in)
        for (int s0 = lane; s0 < a.splits; s0 += kAtOnce * kLanes) {
            float2 u[kAtOnce];
            float4 y[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int s = min(s0 + n * kLanes, a.splits - 1);
                u[n] = *reinterpret_cast<const float2 *>(ms + 2 * (s * rows + at));
                y[n] = *reinterpret_cast<const float4 *>(a.part + (s * rows + at) * a.D + e);
            }
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n)
                if (s0 + n * kLanes < a.splits) p.join(u[n].x, u[n].y, y[n]);
        }
    if constexpr (kLanes > 1) {
        parts[threadIdx.x] = p;
        __syncthreads();
        if (lane) return;
#pragma unroll
        for (int n = 1; n < kLanes; ++n) {
            const Partial &o = parts[threadIdx.x + 32 * n];
            p.join(o.most, o.sum, o.x);
        }
    }
    if (!in) return;
    const int pair = (int)(at / a.R), row = (int)(at % a.R), seq = pair / a.Hk, head = pair % a.Hk, t = row / a.G, g = row % a.G;
    const int64_t token = a.shared ? t : (int64_t)seq * a.Lq + t;
    const float f = p.sum == 0.0f ? 0.0f : 1.0f / p.sum;
    typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf4 *>(a.o + ((token * a.Hk + head) * a.G + g) * a.D + e) =
        bf4{(__bf16)(p.x.x * f), (__bf16)(p.x.y * f), (__bf16)(p.x.z * f), (__bf16)(p.x.w * f)};
}

// The mask as bits: a wave takes kMaskKeys keys of a row, four bytes a lane at once where the rows are
// aligned to that (kWide), else one.
constexpr int kMaskKeys = 1024;
template <bool kWide>
__global__ __launch_bounds__(256) void attn_mask_kernel(const uint8_t *mask, int64_t mask_seq, int64_t mask_row, int64_t rows,
                                                        int Lk, int blocks, uint64_t *words) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), seq = blockIdx.z;
    if (row >= rows) return;
    const auto p = global(mask + seq * mask_seq + row * mask_row);
    const int first = blockIdx.y * kMaskKeys;
    uint64_t mine = 0;  // lane n: word n
    if constexpr (kWide) {
        constexpr int kLoads = kMaskKeys / 256;
        uint32_t u[kLoads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int key = first + 256 * n + 4 * lane;
            u[n] = 0;
            if (key + 4 <= Lk)
                u[n] = *(const __attribute__((address_space(1))) uint32_t *)(p + key);
            else
                for (int i = 0; key + i < Lk; ++i) u[n] |= (uint32_t)p[key + i] << (8 * i);
        }
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            // a bit for every byte that is not 0, the four in a row; then the words of 16 lanes
            uint32_t x = ((u[n] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu | u[n]) >> 7 & 0x01010101u;
            x = (x | x >> 7 | x >> 14 | x >> 21) & 15u;
            uint64_t w = (uint64_t)x << (4 * (lane & 15));
            uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32);
            auto join = [](uint32_t v) {
                v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
                v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
                v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false);
                return v | (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false);
            };
            lo = join(lo);
            hi = join(hi);
            w = (uint64_t)(uint32_t)__shfl((int)hi, (lane & 3) * 16) << 32 | (uint32_t)__shfl((int)lo, (lane & 3) * 16);
            mine = lane / 4 == n ? w : mine;
        }
    } else {
        constexpr int kLoads = kMaskKeys / 64;
        uint8_t u[kLoads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int key = first + 64 * n + lane;
            u[n] = key < Lk ? p[key] : 0;
        }
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const uint64_t w = __ballot(u[n] != 0);
            mine = lane == n ? w : mine;
        }
    }
    const int block = first / kKeys + lane;
    if (lane < kMaskKeys / kKeys && block < blocks) global(words)[(seq * blocks + block) * rows + row] = mine;
}

// --------------------------------------------------------------- host

// Kernels by head size, and by rows: tiles of 32 a wave, waves over rows, waves over keys.
using AttnFn = void (*)(Attn);
template <int RT, int kR, int kK>
AttnFn attn_build(int64_t D) {
    return D <= 64   ? attn_kernel<4, 2, RT, kR, kK>
           : D <= 80 ? attn_kernel<5, 3, RT, kR, kK>
           : D <= 96 ? attn_kernel<6, 3, RT, kR, kK>
                     : attn_kernel<8, 4, RT, kR, kK>;
}
struct Shape {
    int rows, waves, keys;
    AttnFn (*build)(int64_t);
};
const Shape kShapes[] = {
    {32, 1, 1, attn_build<1, 1, 1>},
    {128, 4, 1, attn_build<1, 4, 1>},
    {128, 8, 2, attn_build<1, 4, 2>},
};

struct Plan {
    const Shape *shape;
    int64_t pairs, R, tiles, splits;
    int64_t word_seqs, word_rows, blocks;
    int64_t words, part;  // bytes
};

int check_sizes(const s3d8_cross_attention_args &a) {
    if (a.B <= 0 || a.Lq <= 0 || a.Lk <= 0 || a.heads <= 0 || a.kv_heads <= 0 || a.D <= 0)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (a.B > 65535 || a.Lq > 1 << 24 || a.Lk > 1 << 24 || a.heads > 4096)
        return s3d8::fail(S3D8_ERR_SHAPE, "more than 65535 sequences, 2^24 tokens or keys or 4096 heads are not supported");
    if (a.D % 16 || a.D > 128) return s3d8::fail(S3D8_ERR_SHAPE, "heads must be a multiple of 16 up to 128");
    if (a.heads % a.kv_heads) return s3d8::fail(S3D8_ERR_SHAPE, "heads must be a multiple of kv_heads");
    if (a.B * a.Lq * a.heads > 1 << 30) return s3d8::fail(S3D8_ERR_SHAPE, "B Lq heads over 2^30 is not supported");
    return S3D8_OK;
}

Plan plan(const s3d8_cross_attention_args &a, int cus) {
    Plan p{};
    const int64_t G = a.heads / a.kv_heads;
    p.pairs = (a.shared ? 1 : a.B) * a.kv_heads;
    p.R = (a.shared ? a.B * a.Lq : a.Lq) * G;
    p.blocks = (a.Lk + kKeys - 1) / kKeys;
    const char *force = getenv("ATTN_SHAPE");
    p.shape = force ? &kShapes[atoi(force)] : p.R <= 96 ? &kShapes[0] : p.pairs * ((p.R + 127) / 128) > cus ? &kShapes[1] : &kShapes[2];
    p.tiles = (p.R + p.shape->rows - 1) / p.shape->rows;
    const int64_t groups = p.pairs * p.tiles, most = p.shape->waves == 1 ? p.blocks : p.blocks / (4 * p.shape->keys);
    const int64_t slots = p.shape->keys == 1 ? 2 * cus : cus;
    p.splits = std::max<int64_t>(1, std::min<int64_t>({slots / groups, most, kMaxSplits}));
    if (const char *f = getenv("ATTN_SPLITS")) p.splits = atoi(f);
    if (a.mask) {
        p.word_seqs = a.mask_seq ? a.B : 1;
        p.word_rows = a.mask_row ? a.Lq : 1;
        p.words = (p.word_seqs * p.word_rows * p.blocks * 8 + 15) / 16 * 16;
    }
    if (p.splits > 1) p.part = p.splits * p.pairs * p.R * (a.D + 2) * 4;
    return p;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" {

int64_t s3d8_cross_attention_workspace_bytes(const s3d8_cross_attention_args *args, int32_t num_cus) {
    if (!args || num_cus <= 0 || check_sizes(*args)) return -1;
    const Plan p = plan(*args, num_cus);
    s3d8::clear_error();
    return p.words + p.part;
}

int32_t s3d8_cross_attention(const s3d8_cross_attention_args *args, void *stream) {
    if (!args || !args->q || !args->k || !args->v || !args->o) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    const s3d8_cross_attention_args &a = *args;
    int rc = check_sizes(a);
    if (rc) return rc;
    if ((a.xq != nullptr) != (a.xs != nullptr)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "xq and xs go together");
    if (!(a.scale > 0.0f && a.scale <= 0x1p100f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "scale must be positive (at most 2^100)");
    if (a.xq && a.heads * a.D > 65536) return s3d8::fail(S3D8_ERR_SHAPE, "codes of rows over 65536 are not supported");
    if (a.xq && a.B * a.Lq > 1 << 19) return s3d8::fail(S3D8_ERR_SHAPE, "codes of more than 524288 rows are not supported");
    const int64_t lim = int64_t(1) << 40;
    for (int64_t s : {a.q_seq, a.q_row, a.q_head, a.k_seq, a.k_row, a.k_head, a.v_seq, a.v_row, a.v_head}) {
        if (s < 0 || s > lim) return s3d8::fail(S3D8_ERR_INVALID_ARG, "strides must not be negative (and at most 2^40)");
        if (s % 8) return s3d8::fail(S3D8_ERR_ALIGN, "strides must be multiples of 8");
    }
    if (a.Lk > 1 && (a.k_row < a.D || a.v_row < a.D || a.k_row >= 1 << 23 || a.v_row >= 1 << 23))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "k_row and v_row must be at least D and below 2^23");
    if (a.mask && (a.mask_seq < 0 || a.mask_row < 0 || a.mask_seq > lim || a.mask_row > lim))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "mask strides must not be negative (and at most 2^40)");
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.o, 16) || !aligned(a.xq, 16) ||
        !aligned(a.workspace, 16))
        return s3d8::fail(S3D8_ERR_ALIGN, "q, k, v, o, xq and workspace must be 16-byte aligned");
    if (!aligned(a.kv_lens, 4) || !aligned(a.xs, 4)) return s3d8::fail(S3D8_ERR_ALIGN, "kv_lens and xs must be 4-byte aligned");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    const Plan p = plan(a, cus);
    if (p.words + p.part > 0 && (!a.workspace || a.workspace_bytes < p.words + p.part))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "workspace smaller than s3d8_cross_attention_workspace_bytes");
    if (p.pairs * p.tiles * p.splits * 64 * p.shape->waves >= int64_t(1) << 32)
        return s3d8::fail(S3D8_ERR_SHAPE, "more than 2^32 threads are not supported");
    Attn d{};
    d.q = a.q;
    d.k = a.k;
    d.v = a.v;
    d.lens = a.kv_lens;
    d.o = a.o;
    d.part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + p.words);
    d.q_seq = a.q_seq;
    d.q_row = a.q_row;
    d.q_head = a.q_head;
    d.k_seq = a.k_seq;
    d.k_row = a.Lk > 1 ? a.k_row : a.D;
    d.k_head = a.k_head;
    d.v_seq = a.v_seq;
    d.v_row = a.Lk > 1 ? a.v_row : a.D;
    d.v_head = a.v_head;
    d.Lq = (int)a.Lq;
    d.Lk = (int)a.Lk;
    d.G = (int)(a.heads / a.kv_heads);
    d.Hk = (int)a.kv_heads;
    d.D = (int)a.D;
    d.R = (int)p.R;
    d.pairs = (int)p.pairs;
    d.tiles = (int)p.tiles;
    d.splits = (int)p.splits;
    d.shared = a.shared != 0;
    d.scale = a.scale * 0x1.715476p+0f;
    if (a.mask) {
        uint64_t *words = static_cast<uint64_t *>(a.workspace);
        d.words = words;
        d.word_seq = a.mask_seq ? p.blocks * p.word_rows : 0;
        d.word_block = p.word_rows;
        d.word_row = a.mask_row ? 1 : 0;
        const bool wide = aligned(a.mask, 4) && a.mask_seq % 4 == 0 && a.mask_row % 4 == 0;
        hipLaunchKernelGGL(wide ? attn_mask_kernel<true> : attn_mask_kernel<false>,
                           dim3((unsigned)((p.word_rows + 3) / 4), (unsigned)((a.Lk + kMaskKeys - 1) / kMaskKeys),
                                (unsigned)p.word_seqs),
                           dim3(256), 0, (hipStream_t)stream, a.mask, a.mask_seq, a.mask_row, p.word_rows, (int)a.Lk,
                           (int)p.blocks, words);
    }
    hipLaunchKernelGGL(p.shape->build(a.D), dim3((unsigned)(p.pairs * p.tiles * p.splits)),
                       dim3((unsigned)(64 * p.shape->waves)), 0, (hipStream_t)stream, d);
    if (p.splits > 1) {
        const int64_t rows = p.pairs * p.R;
        if (p.splits > 4)
            hipLaunchKernelGGL(attn_join_kernel<8>, dim3((unsigned)rows), dim3(256), 0, (hipStream_t)stream, d);
        else
            hipLaunchKernelGGL(attn_join_kernel<1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, (hipStream_t)stream, d);
    }
    if (a.xq) s3d8::codes_of_rows(a.o, a.B * a.Lq, a.heads * a.D, a.xq, a.xs, cus, stream);
    return s3d8::launch_status();
}

}  // extern "C"
