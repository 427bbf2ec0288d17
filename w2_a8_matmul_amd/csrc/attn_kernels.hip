// Attention of query tokens to an encoder's states, for gfx950: with p_j = exp(scale q.k_j)
//   o = sum_j p_j v_j / sum_j p_j
// in one pass over the keys, with a running maximum taken off the scores.
//
// The query tokens and heads that read one key head are the rows of one problem, so each key
// and value is fetched once for all of them, and an 8-fold group decodes at the cost of one head.
// Scores are computed transposed, S = K Q^T, in 32 x 32 x 16 products: a row's scores are
// then in the registers of two lanes, its maximum and sum need one step between lanes, and
// the rounded p are the operand of O^T = V^T P^T as they stand; LDS transposes the values as it reads
// them.  Keys and values go from memory to LDS without registers, two blocks of each in
// turn.  p is rounded to bf16, the type of the product with v; the sum takes the rounded p, so
// that the weights of the values add up to 1.  Scores, maximum, sums and o are fp32.
//
//   mask  the mask as bits, 64 keys a word (6.9 us for 2048 x 6404 bytes)
//   attn  tiles of rows, each over all keys or a part of them
//   join  the parts' sums
//
// Few rows are bound by the reading of keys and values: 8 sequences of one token, 32 heads on 8 of 128,
// 38 thousand states in all, 157 MB: 36 to 38 us, 4.1 to 4.4 TB/s (a copy reaches 5.1).  Many rows are bound by the
// matrix products and the exponentials beside them, of which each takes a SIMD about as
// long: 2048 tokens on 6404 states, 215 GFLOP: 201 to 205 us, 1.05 PFLOP/s (a large product by itself 1.28);
// vector instructions in a product's shadow are not free (a 32 x 32 product 36 ticks, six fmas
// 33, both together 50).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kKeys = 64;       // keys in a word of the mask
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

// Of two bf16 numbers in a word: those that are finite, and a code of each of the others, 1 for
// infinity, 32 for minus infinity and 1024 for NaN: sums of 16 codes tell which were among them.
__device__ __forceinline__ void take_apart(uint32_t w, uint32_t &finite, uint32_t &codes) {
    finite = codes = 0;
#pragma unroll
    for (int n = 0; n < 32; n += 16) {
        const uint32_t x = w >> n & 0xFFFFu;
        const bool is = (x & 0x7F80u) != 0x7F80u;
        finite |= (is ? x : 0) << n;
        codes |= (is ? 0 : x & 0x7Fu ? 0x4480u : x & 0x8000u ? 0x4200u : 0x3F80u) << n;
    }
}
__device__ __forceinline__ float with_codes(float x, int codes) {
    if (codes == 0) return x;
    const bool above = codes & 31, below = codes >> 5;  // (NaN: below, and not minus infinity alone)
    return x + (codes >> 10 || (above && below) ? NAN : above ? INFINITY : -INFINITY);
}

// A workgroup of kR x kK waves: kR over rows, 32 each; kK over keys, each on every kK-th block of
// the split's keys with tiles in LDS of its own, joined at the end.  KB keys in a block.  LDS and
// registers hold two workgroups on a CU, two waves a SIMD, so that one wave's vector work runs beside
// the other's products: 64 rows a wave and one wave a SIMD took 260 us where this takes 205
// (2048 tokens on 6404 states), three waves a SIMD spill.  The blocks that no row of a tile sees are left out
// of the wave's list before the loop: a branch around them in the loop keeps the next block's
// scores from being computed beside this block's exponentials, and spilled (1540 us).
template <int NK, int ND, int kR, int kK, int KB>
__global__ __launch_bounds__(64 * kR * kK, 2) void attn_kernel(const Attn a) {
    constexpr int Dp = 32 * ND;      // entries of a row in LDS
    constexpr int CPR = Dp / 8;
    constexpr int kTile = KB * CPR;  // chunks
    constexpr int KT = KB / 32, kScores = KT * NK, kSums = KB / 16 * ND;  // products for a block
    constexpr int kCopies = kTile / 64 / kR;
    static_assert(16 * NK <= Dp && kTile % (64 * kR) == 0, "");
    __shared__ __attribute__((aligned(1024))) uint4 tiles[kK][2][2][kTile];  // keys and values, two blocks of each
    __shared__ uint64_t seen[kListed / 64];
    __shared__ uint16_t list[kListed];
    __shared__ int again;  // sums are formed twice

    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), wr = wave % kR, wk = wave / kR;
    const int pair = (int)blockIdx.x % a.pairs, rest = (int)blockIdx.x / a.pairs;
    const int tile = rest % a.tiles, split = rest / a.tiles;
    const int seq = pair / a.Hk, head = pair % a.Hk;

    int len = a.lens ? global(a.lens)[a.shared ? 0 : seq] : a.Lk;
    len = max(0, min(len, a.Lk));
    const int blocks = (len + KB - 1) / KB;
    const int begin = (int)((int64_t)blocks * split / a.splits), end = (int)((int64_t)blocks * (split + 1) / a.splits);

    // this lane's row (past the last: the last again, not stored)
    const int row = (tile * kR + wr) * kRows + col, rr = min(row, a.R - 1), t = rr / a.G;
    const int b = a.shared ? t / a.Lq : seq, i = a.shared ? t % a.Lq : t, q_head = head * a.G + rr % a.G;
    const int64_t q_at = b * a.q_seq + i * a.q_row + q_head * a.q_head, word_at = b * a.word_seq + i * a.word_row;
    bf8 qf[NK];
#pragma unroll
    for (int s = 0; s < NK; ++s) {
        v4u u = {0, 0, 0, 0};
        if (16 * s + 8 * h < a.D) u = *global(reinterpret_cast<const v4u *>(a.q + q_at + 16 * s + 8 * h));
        qf[s] = __builtin_bit_cast(bf8, u);
    }

    // the lane's part of each copy of a tile into LDS
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
        const int rows = min(KB, len - block * KB) - 1;
        const v4i r = rsrc_words(p + (int64_t)block * KB * stride, block < end ? (uint32_t)(rows * stride + a.D) * 2 : 0);
#pragma unroll
        for (int n = 0; n < kCopies; ++n) load_to_lds16_so(S3D8_LDS_OFFSET(to + (wr + n * kR) * 64), off[n], 0, r);
    };
    auto copy_keys = [&](int block, int slot) { copy(kp, a.k_row, block, tiles[wk][0][slot], koff); };
    auto copy_values = [&](int block, int slot) { copy(vp, a.v_row, block, tiles[wk][1][slot], voff); };

    // the mask's bits of a block, of 64 keys a word
    // (shifted where they are used, a step later: a shift at the load waits for it)
    auto load_word = [&](int64_t at, int block) { return global(a.words)[at + block * KB / kKeys * a.word_block]; };
    auto bits_of = [&](uint64_t word, int block) { return word >> (block * KB % kKeys); };  // the block's: the first KB
    constexpr uint64_t kAll = KB == 64 ? ~0ull : (1ull << (KB % 64)) - 1;

    // With a mask, the blocks that any row of the tile sees, by the words of the tile's tokens: a lane a
    // block, a wave every kR kK-th token.
    int count = end - begin;
    const bool sparse = a.words && count <= kListed;
    if (sparse) {
        for (int n = threadIdx.x; n < kListed / 64; n += 64 * kR * kK) seen[n] = 0;
        __syncthreads();
        const int r0 = tile * kR * kRows, t0 = r0 / a.G, t1 = min(r0 + kR * kRows - 1, a.R - 1) / a.G;
        for (int n = 0; n < count; n += 64) {
            const int block = min(begin + n + lane, end - 1);
            uint64_t any = 0;
#pragma unroll 4
            for (int t = t0 + wave; t <= t1; t += kR * kK)
                any |= load_word((a.shared ? t / a.Lq : seq) * a.word_seq + (a.shared ? t % a.Lq : t) * a.word_row, block);
            const uint64_t bits = __ballot((bits_of(any, block) & kAll) != 0 && n + lane < count);
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

    f16v acc[ND];
    float most = -FLT_MAX, sum = 0.0f;  // of scaled scores, in powers of 2; this lane's part of the sum
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;

    // a score operand (32 keys, 16 entries) and a value operand (32 entries, 16 keys; transposed by the
    // read: entry by lane, four keys in a row) of a block
    auto key_operand = [&](int slot, int i) {
        const int n = i / KT, r = i % KT * 32 + col;
        return *reinterpret_cast<const bf8 *>(reinterpret_cast<const char *>(tiles[wk][0][slot]) +
                                              (r * CPR + key_place<CPR>(2 * n + h, r)) * 16);
    };
    auto value_operand = [&](int slot, int i) {
        const int n = i / ND, d = i % ND;
        struct Two {
            s4 x[2];
        } two;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 16 * n + 8 * j + 4 * h + ((lane & 15) >> 2);
            const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            two.x[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s4 *)(reinterpret_cast<const char *>(tiles[wk][1][slot]) +
                                                         (r * CPR + value_place<CPR>(c, r)) * 16 + 8 * (lane & 1)));
        }
        return __builtin_bit_cast(bf8, two);
    };
    auto word_of = [&](int block) { return a.words && block < end ? load_word(word_at, block) : ~0ull; };
    auto inside = [&](int block) {  // the bits of the keys that exist
        const int n = block < end ? len - block * KB : 0;
        return n < KB ? (1ull << max(n, 0)) - 1 : kAll;
    };
    auto most_of = [&](const f16v(&s)[KT]) {
        float m = s[0][0];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) m = fmaxf(m, s[kt][r]);
        return m;
    };

    // Scores are transposed: key by register, row by lane.  Block n is weighed and added while the
    // scores of the next block are computed: their products run beside the exponentials, and the
    // largest of them is found beside the products with the values.
    const int steps = (count + kK - 1) / kK;
    if (threadIdx.x == 0) again = 0;  // (read after the steps' barriers)
    if (steps > 0) {
        int block = block_at(0), next = block_at(1);
        uint64_t word = word_of(block), next_word = word_of(next);
        copy_keys(block, 0);
        copy_values(block, 0);
        wait_vmcnt_barrier<0>();
        copy_keys(next, 1);
        f16v s[KT], t[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kt][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < kScores; ++i)
            s[i % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_operand(0, i), qf[i / KT], s[i % KT], 0, 0, 0);
        float m = most_of(s);

        auto step = [&](int n, int slot, f16v(&s)[KT], f16v(&t)[KT]) {
            const int later = block_at(n + 2), other = slot ^ 1;
            wait_vmcnt_barrier<0>();
            const uint64_t bits = bits_of(word, block) & inside(block);
            word = next_word;
            next_word = word_of(later);
            copy_keys(later, slot);  // this block's keys were read a step ago, the last one's values too
            copy_values(next, other);
            block = next;
            next = later;
            if (__ballot(bits != kAll)) {
                const uint64_t mine = bits >> (4 * h);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[kt][r] = (uint32_t)(mine >> (32 * kt)) >> (8 * (r / 4) + r % 4) & 1 ? s[kt][r] : -INFINITY;
                m = most_of(s);
            }
            m = halves_max(m) * a.scale;
            if (__ballot(m > most + kSlack)) {
                m = fmaxf(most, m);
                const float f = __builtin_amdgcn_exp2f(most - m);
                most = m;
                sum *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] *= f;
            }
            constexpr int kAhead = 4;  // operands in flight
            bf8 operand[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) operand[i] = key_operand(other, i);
            uint32_t pf[KB / 4];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 16; ++r) t[kt][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < kScores; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                t[i % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand[i % kAhead], qf[i / KT], t[i % KT], 0, 0, 0);
                operand[i % kAhead] = i + kAhead < kScores ? key_operand(other, i + kAhead) : value_operand(slot, i + kAhead - kScores);
#pragma unroll
                for (int e = i * (KB / 4) / kScores; e < (i + 1) * (KB / 4) / kScores; ++e) {
                    bf2 two;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        two[x] = (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 8][2 * (e % 8) + x], a.scale, -most));
                    sum = __builtin_amdgcn_fdot2_f32_bf16(two, bf2{(__bf16)1.0f, (__bf16)1.0f}, sum, false);
                    pf[e] = __builtin_bit_cast(uint32_t, two);
                }
            }
            m = t[0][0];
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                const uint4 p = make_uint4(pf[i / ND * 4], pf[i / ND * 4 + 1], pf[i / ND * 4 + 2], pf[i / ND * 4 + 3]);
                acc[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand[(i + kScores) % kAhead], __builtin_bit_cast(bf8, p),
                                                                      acc[i % ND], 0, 0, 0);
                if (i + kAhead < kSums) operand[(i + kScores) % kAhead] = value_operand(slot, i + kAhead);
#pragma unroll
                for (int e = i * (KB / 2) / kSums; e < (i + 1) * (KB / 2) / kSums; ++e) m = fmaxf(m, t[e / 16][e % 16]);
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
    if (a.words && steps > 0) {
        // A hidden key has p = 0, but the product with an infinite or NaN value of it is NaN. Sums that are
        // not finite are formed again over the same p, from the finite values, and by a product of the
        // keys that a row sees with codes of the other values, which of those are among them: the bits are
        // those of a call whose hidden values are 0. (A row whose scores have a NaN is NaN: it stays.) One step
        // after the other, copies a step ahead: 1.0 ms in all where a mask of images on 2048 x 6404 takes 0.2 (2.0
        // where no value is finite).
        float z = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) z = __builtin_fmaf(acc[d][r], 0.0f, z);
        uint64_t lost = __ballot(z != z && row < a.R);
        const uint64_t none = __ballot(sum != sum);
        lost = (lost | lost >> 32) & ~(none | none >> 32) & 0xFFFFFFFFull;
        if (lost && lane == 0) again = 1;
        __syncthreads();
        if (again) {  // (the workgroup's: its waves share tiles)
            const bool mine = lost >> col & 1;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] = mine ? 0.0f : acc[d][r];
            float top = -FLT_MAX;  // the running maximum as it was
            copy_keys(block_at(0), 0);
            copy_values(block_at(0), 0);
            for (int n = 0; n < steps; ++n) {
                const int slot = n & 1, block = block_at(n), next = block_at(n + 1);
                const uint64_t bits = bits_of(word_of(block), block) & inside(block);
                wait_vmcnt_barrier<0>();
                copy_keys(next, slot ^ 1);  // read by all a step ago
                copy_values(next, slot ^ 1);
                if (!lost) continue;
                f16v s[KT];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[kt][r] = 0.0f;
#pragma unroll
                for (int i = 0; i < kScores; ++i)
                    s[i % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_operand(slot, i), qf[i / KT], s[i % KT], 0, 0, 0);
                // (the bits of register r, and of the one after it)
                auto sees = [&](int kt, int r) { return (uint32_t)(bits >> (4 * h + 32 * kt)) >> (8 * (r / 4) + r % 4); };
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[kt][r] = sees(kt, r) & 1 ? s[kt][r] : -INFINITY;
                float m = halves_max(most_of(s)) * a.scale;
                if (__ballot(m > top + kSlack)) {
                    m = fmaxf(top, m);
                    const float f = mine ? __builtin_amdgcn_exp2f(top - m) : 1.0f;
                    top = m;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[d][r] *= f;
                }
                // p, and 1 for a key that is seen: of the lost rows, the others' sums stay
                uint32_t pf[KB / 4], one[KB / 4];
#pragma unroll
                for (int e = 0; e < KB / 4; ++e) {
                    bf2 two;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        two[x] = (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 8][2 * (e % 8) + x], a.scale, -top));
                    const uint32_t which = sees(e / 8, 2 * (e % 8));
                    pf[e] = mine ? __builtin_bit_cast(uint32_t, two) : 0;
                    one[e] = mine ? (which & 1) * 0x3F80u | (which >> 1 & 1) * 0x3F800000u : 0;
                }
#pragma unroll
                for (int i = 0; i < kSums; ++i) {
                    const int e = i / ND * 4;
                    const v4u v = __builtin_bit_cast(v4u, value_operand(slot, i));
                    v4u finite, codes;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t f, c;
                        take_apart(v[x], f, c);
                        finite[x] = f;
                        codes[x] = c;
                    }
                    acc[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf8, finite), __builtin_bit_cast(bf8, make_uint4(pf[e], pf[e + 1], pf[e + 2], pf[e + 3])),
                        acc[i % ND], 0, 0, 0);
                    if (!__ballot((codes[0] | codes[1] | codes[2] | codes[3]) != 0)) continue;
                    f16v among;
#pragma unroll
                    for (int r = 0; r < 16; ++r) among[r] = 0.0f;
                    among = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf8, codes), __builtin_bit_cast(bf8, make_uint4(one[e], one[e + 1], one[e + 2], one[e + 3])),
                        among, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i % ND][r] = with_codes(acc[i % ND][r], (int)among[r]);
                }
            }
            wait_vmcnt_barrier<0>();
        }
    }
    sum += __shfl_xor(sum, 32);

    if constexpr (kK > 1) {
        // the waves over keys joined, one after the other, through the tiles' LDS
        float4 *room = reinterpret_cast<float4 *>(tiles) + wr * (64 * (4 * ND + 1));
        static_assert(kR * 64 * (4 * ND + 1) * 16 <= (int)sizeof(tiles), "");
        for (int g = 1; g < kK; ++g) {
            __syncthreads();
            if (wk == g) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        room[(d * 4 + q) * 64 + lane] =
                            make_float4(acc[d][4 * q], acc[d][4 * q + 1], acc[d][4 * q + 2], acc[d][4 * q + 3]);
                room[ND * 4 * 64 + lane] = make_float4(most, sum, 0.0f, 0.0f);
            }
            __syncthreads();
            if (wk == 0) {
                const float4 ms = room[ND * 4 * 64 + lane];
                const float top = fmaxf(most, ms.x), f = __builtin_amdgcn_exp2f(most - top), o = __builtin_amdgcn_exp2f(ms.x - top);
                most = top;
                sum = __builtin_fmaf(f, sum, o * ms.y);
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 x = room[(d * 4 + q) * 64 + lane];
                        acc[d][4 * q] = __builtin_fmaf(f, acc[d][4 * q], o * x.x);
                        acc[d][4 * q + 1] = __builtin_fmaf(f, acc[d][4 * q + 1], o * x.y);
                        acc[d][4 * q + 2] = __builtin_fmaf(f, acc[d][4 * q + 2], o * x.z);
                        acc[d][4 * q + 3] = __builtin_fmaf(f, acc[d][4 * q + 3], o * x.w);
                    }
            }
        }
        if (wk) return;
    }
    if (row >= a.R) return;
    if (a.splits > 1) {
        const int64_t at = ((int64_t)split * a.pairs + pair) * a.R + row;
        const auto p = global(a.part) + at * a.D;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int e = 32 * d + 2 * r + 4 * h;
                const v4f x = {acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]};
                if (e < a.D) *(__attribute__((address_space(1))) v4f *)(p + e) = x;
            }
        if (h == 0) {
            const auto ms = global(a.part) + (int64_t)a.splits * a.pairs * a.R * a.D + 2 * at;
            ms[0] = most;
            ms[1] = sum;
        }
        return;
    }
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const auto o = global(a.o) + (((int64_t)b * a.Lq + i) * a.Hk * a.G + q_head) * a.D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
            const int e = 32 * d + 2 * r + 4 * h;
            const bf4 x = {(__bf16)(acc[d][r] * f), (__bf16)(acc[d][r + 1] * f), (__bf16)(acc[d][r + 2] * f), (__bf16)(acc[d][r + 3] * f)};
            if (e < a.D) *(__attribute__((address_space(1))) bf4 *)(o + e) = x;
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

// The mask as bits: a wave takes kMaskKeys keys of a row, four bytes a lane at once (at any address).
constexpr int kMaskKeys = 1024;
typedef uint32_t u32_any __attribute__((aligned(1)));
__global__ __launch_bounds__(256) void attn_mask_kernel(const uint8_t *mask, int64_t mask_seq, int64_t mask_row, int64_t rows,
                                                        int Lk, int blocks, uint64_t *words) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), seq = blockIdx.z;
    if (row >= rows) return;
    const auto p = global(mask + seq * mask_seq + row * mask_row);
    const int first = blockIdx.y * kMaskKeys;
    uint64_t mine = 0;  // lane n: word n
    constexpr int kLoads = kMaskKeys / 256;
    uint32_t u[kLoads];
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
        const int key = first + 256 * n + 4 * lane;
        u[n] = 0;
        if (key + 4 <= Lk)
            u[n] = *(const __attribute__((address_space(1))) u32_any *)(p + key);
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
    const int block = first / kKeys + lane;
    if (lane < kMaskKeys / kKeys && block < blocks) global(words)[(seq * blocks + block) * rows + row] = mine;
}

// --------------------------------------------------------------- host

// Kernels by head size.
using AttnFn = void (*)(Attn);
template <int kR, int kK, int KB>
AttnFn attn_build(int64_t D) {
    return D <= 64   ? attn_kernel<4, 2, kR, kK, KB>
           : D <= 80 ? attn_kernel<5, 3, kR, kK, KB>
           : D <= 96 ? attn_kernel<6, 3, kR, kK, KB>
                     : attn_kernel<8, 4, kR, kK, KB>;
}

struct Plan {
    bool wide;  // tiles of 128 rows, else 64
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
    // Tiles of 128 rows where there is more than one for every CU, else of 64 (2048 tokens, 32 heads on 1601
    // keys: one of 128 for two CUs 31 us, of 64 for each 26; 2048 on 6404: of 128, two a CU, 205).
    p.wide = p.pairs * ((p.R + 127) / 128) > cus;
    const int64_t rows = p.wide ? 128 : 64;
    p.tiles = (p.R + rows - 1) / rows;
    // The split of the keys with the least estimated time, in us of 128-entry heads: 0.7 for a block of 64
    // keys where a CU has one workgroup, 1.05 where it has two; the join's launch, and the sums it reads
    // (one token on 1601 keys: 23.5 us unsplit, 9.0 in 26; 100 on 1601: 24.1, 17.4 in 4, 21.6 in 8).
    const int64_t groups = p.pairs * p.tiles;
    double best = 1e30;
    for (int64_t s = 1; s <= std::min<int64_t>(p.blocks, kMaxSplits); ++s) {
        const int64_t rounds = (groups * s + 2 * cus - 1) / (2 * cus), blocks = (p.blocks + s - 1) / s;
        const double t = (double)(rounds * blocks) * (groups * s <= cus ? 0.7 : 1.05) +
                         (s > 1 ? 3.0 + 2.9e-6 * (double)(p.pairs * p.R * a.D * s) : 0.0);
        if (t < best) {
            best = t;
            p.splits = s;
        }
        if (p.wide) break;
    }
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
    if (p.pairs * p.tiles * p.splits * 256 >= int64_t(1) << 32)
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
        hipLaunchKernelGGL(attn_mask_kernel,
                           dim3((unsigned)((p.word_rows + 3) / 4), (unsigned)((a.Lk + kMaskKeys - 1) / kMaskKeys),
                                (unsigned)p.word_seqs),
                           dim3(256), 0, (hipStream_t)stream, a.mask, a.mask_seq, a.mask_row, p.word_rows, (int)a.Lk,
                           (int)p.blocks, words);
    }
    const AttnFn fn = p.wide ? attn_build<4, 1, 64>(a.D) : attn_build<2, 2, 32>(a.D);
    hipLaunchKernelGGL(fn, dim3((unsigned)(p.pairs * p.tiles * p.splits)), dim3(256), 0, (hipStream_t)stream, d);
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
