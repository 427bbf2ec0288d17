// The choice of the next token from rows of logits, for gfx950: of the tokens that top-k, top-p
// and min-p keep, the one at which the running sum of the weights W(i) = exp((l_i - max l) / T), in the
// order of the index, passes u times their sum.
//
// Weights are whole numbers (2^44 times the exponential, rounded), so that sums of them do
// not depend on their order: workgroups add them with atomics as they come, and the token is
// the same on every run.  A row is cut into parts, so that few rows still fill the device:
//   part  the largest logit of each part; with a top-k of at most 1024 also the part's
//         candidates, in one read of the logits (below);
//   bins  without a top-k: sums of the weights by the logit's distance from the largest, in
//         steps of a 64th of temperature, and so the step in which top-p ends;
//   step  the tokens of that step, and the kept weight of each segment of the row;
//   row   the rest for one row: the exact end of top-k and top-p among the few that are left,
//         min-p, and the token at the random number, in the list of candidates or in the one segment
//         that holds it.
// With a top-k alone the launches are `part` and `row`; a vocabulary of at most 3584 tokens is listed
// by `row` itself, which is then the only one.  Rows for which a list is too short (a top-k over
// 1024, thousands of equal logits) are done by `row` alone, digit by digit of the tokens'
// order, in up to a dozen reads of the row (464 us for 5000 of one row's 128256 tokens).
//
// Many rows with a top-k are bound by the one read: 512 rows of 128256 fp32, 263 MB, k = 50: `part` 70 to
// 74 us (51 without the lists, 5.1 TB/s as a copy), `row` 12.  Without a top-k `bins` and `step` are bound by
// the exponentials in 64 bits, one a token: 111 and 146 us beside the 50 of `part`.  Few rows are bound
// by the chain of steps in one workgroup, each of which waits for the last: one row, k = 50: 8 us
// each of `part` and `row`.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

constexpr int64_t kMaxVocabulary = 1 << 18;  // 2^18 weights of 2^44 stay below 2^63
constexpr int64_t kMaxRows = 1 << 19;
constexpr int64_t kRowsAtOnce = 1024;        // rows of one set of launches (bounds the workspace)
constexpr int kT = 512;                      // threads of every workgroup; vectors of a segment
constexpr int kMaxTopK = 1024;
constexpr int kListed = 3584;                // candidates of a part, tokens of a step, a vocabulary that is listed whole
constexpr int kRound = 4;                    // segments that are read at once
constexpr int kDigit = 11, kBins = 1 << kDigit;
constexpr int kSteps = 64;                   // bins per unit of (largest logit - logit) / temperature
constexpr int kIndexBits = 18;
constexpr int kOrderBits = 32 + kIndexBits;
constexpr uint32_t kNothing = 0x007FFFFFu;   // order_key(-infinity)
constexpr uint32_t kTooMany = ~0u;
constexpr int kMaxParts = 32;
constexpr int kTops = 4096;                  // tops of a row that are looked at
constexpr int kFewest = 128;                 // tokens that are compared with one another
constexpr int kFewTokens = 2 * kT;           // tokens that are sorted

// fp32 values as whole numbers that order like them (-0 as 0, NaN as -infinity).
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return l != l ? kNothing : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// Place of a token in the order of falling logits, then rising index.
__device__ __forceinline__ uint64_t place(uint32_t key, uint32_t index) {
    return (uint64_t)(~key) << kIndexBits | index;
}
__device__ __forceinline__ uint32_t place_key(uint64_t p) { return ~(uint32_t)(p >> kIndexBits); }
__device__ __forceinline__ uint32_t place_index(uint64_t p) { return (uint32_t)p & ((1u << kIndexBits) - 1); }

// What a workgroup reads.  Arrays of the workspace by row and part.
struct Job {
    s3d8_sample_args a;
    bool direct;          // the row alone, its tokens all listed
    int parts, cuts;      // parts of a row; the same of the launches that take every weight
    int segments;         // room for segment sums
    uint64_t *first;      // [M][parts] the first place of each part
    uint32_t *counts;     // [M][parts] candidates listed, or kTooMany; NULL: no row has a top-k within kMaxTopK
    uint64_t *lists;      // [M][parts][kListed]
    uint32_t *tops;       // [M][parts][groups] the largest key of each group of kT / groups threads
    int groups;           // a power of two, 8 to 256
    uint64_t *bins;       // [M][kBins], or NULL: every row has one
    uint64_t *step;       // [M][kListed] the places of the step in which top-p ends
    uint64_t *sums;       // [M][segments] kept weight of a segment, without that step
    uint64_t *ends;       // [M][2] the step, the weight that is left for it
    uint32_t *steps;      // [M] tokens in `step`
};

// The limits of a row.
struct Limits {
    double t, rt;
    float top_p, min_p;
    int k;        // 0: all
    bool greedy;  // the largest logit alone
    __device__ __forceinline__ Limits(const s3d8_sample_args &a, int64_t r) {
        const float t32 = a.temperature ? global(a.temperature)[r] : a.temperature_all;
        greedy = !(t32 > 0.0f);  // (NaN too)
        t = greedy ? 1.0 : (double)fminf(t32, 0x1p100f);
        rt = 1.0 / t;
        k = a.top_k ? global(a.top_k)[r] : a.top_k_all;
        if (k < 0 || k >= a.V) k = 0;
        top_p = fmaxf(a.top_p ? global(a.top_p)[r] : a.top_p_all, 0.0f);
        min_p = fminf(fmaxf(a.min_p ? global(a.min_p)[r] : a.min_p_all, 0.0f), 1.0f);
    }
    __device__ __forceinline__ bool listed() const { return !greedy && k > 0 && k <= kMaxTopK; }
    __device__ __forceinline__ bool binned() const { return !greedy && k == 0; }
    __device__ __forceinline__ uint64_t least() const { return (uint64_t)ceil((double)min_p * 0x1p44); }
    __device__ __forceinline__ uint64_t end(uint64_t sum) const {
        return max(1ull, (unsigned long long)ceil((double)top_p * (double)sum));
    }
};

// W = rne(2^44 exp((l - m) / t)).  The quotient is l - m times 1 / t with its
// remainder's share, so that it is rounded once; below -60 the weight is 0.
struct Weights {
    uint32_t top;
    double m, t, rt;
    __device__ __forceinline__ Weights(uint32_t top, const Limits &l) : top(top), m((double)key_value(top)), t(l.t), rt(l.rt) {}
    __device__ __forceinline__ double exponent(float l) const {  // NaN where l is infinite
        const double d = (double)l - m, x = d * rt;
        return __builtin_fma(__builtin_fma(-x, t, d), rt, x);
    }
    __device__ __forceinline__ uint64_t of(double x) const {
        if (!(x > -60.0)) return 0;
        const Exp e = exp_parts(x);
        const double s = e.two_n * 0x1p44;
        // 2^52 added rounds to a whole number, which the sum's low bits then are
        return (uint64_t)__double_as_longlong(__builtin_fma(s, e.less_one, s) + 0x1p52) & ((1ull << 52) - 1);
    }
    __device__ __forceinline__ uint64_t operator()(uint32_t key) const {
        return key == top ? 1ull << 44 : key <= kNothing ? 0 : of(exponent(key_value(key)));
    }
    // the same of a logit, and the bin of the distance from the largest one (the last: no weight, NaN too)
    __device__ __forceinline__ int bin(float l, double &x) const {
        x = (double)l == m ? 0.0 : exponent(l);
        return x > -(double)kBins / kSteps ? min((int)(x * -(double)kSteps), kBins - 1) : kBins - 1;
    }
    __device__ __forceinline__ uint64_t at(float l, double x) const { return (double)l == m ? 1ull << 44 : of(x); }
    // Logits below this one are in bins past `last`, and those of the last bin have no weight: 2^44 exp(-32) is
    // less than half. One bin and 2^-20 of the value are left for rounding.
    __device__ __forceinline__ float cut(int last) const {
        const double c = m - t * (double)(min(last, kBins) + 2) * (1.0 / kSteps);
        const float f = (float)(c - __builtin_fabs(c) * 0x1p-20);
        return f == f ? f : -INFINITY;
    }
};

// A row of logits as slots of 16 aligned bytes: slot 0 what comes before the first of them, slots 1
// to n, and slot n + 1 what is left.  Segment s is the slots kT s and following.
template <bool kBF>
struct Row {
    static constexpr int kV = kBF ? 8 : 4;
    const char *p;
    int V, head, n;
    __device__ __forceinline__ Row(const s3d8_sample_args &a, int64_t r)
        : p(static_cast<const char *>(a.logits) + r * a.row * (kBF ? 2 : 4)), V((int)a.V) {
        head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (kBF ? 2 : 4));
        n = (V - head) / kV;
    }
    __device__ __forceinline__ int segments() const { return (n + 2 + kT - 1) / kT; }
    __device__ __forceinline__ int index(int slot) const { return slot == 0 ? 0 : head + (slot - 1) * kV; }
    __device__ __forceinline__ int slot(int index) const { return index < head ? 0 : (index - head) / kV + 1; }
    __device__ __forceinline__ float one(int i) const {
        if constexpr (kBF)
            return bf16_to_f32(global(reinterpret_cast<const uint16_t *>(p))[i]);
        else
            return global(reinterpret_cast<const float *>(p))[i];
    }
    struct Slot {
        v4u u;
        __device__ __forceinline__ float operator[](int j) const {
            return kBF ? __uint_as_float(j & 1 ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16) : __uint_as_float(u[j & 3]);
        }
    };
    // NaN where there is no token
    __device__ __forceinline__ Slot load(int slot) const {
        if (slot >= 1 && slot <= n)
            return Slot{*global(reinterpret_cast<const v4u *>(p + (int64_t)(head + (slot - 1) * kV) * (kBF ? 2 : 4)))};
        const int i = index(slot), end = slot == 0 ? head : slot == n + 1 ? V : i;
        v4u w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (kBF) {
                const auto e = global(reinterpret_cast<const uint16_t *>(p));
                const uint32_t lo = i + 2 * j < end ? e[i + 2 * j] : 0x7FC0u;
                const uint32_t hi = i + 2 * j + 1 < end ? e[i + 2 * j + 1] : 0x7FC0u;
                w[j] = lo | hi << 16;
            } else {
                w[j] = i + j < end ? global(reinterpret_cast<const uint32_t *>(p))[i + j] : 0x7FC00000u;
            }
        }
        return Slot{w};
    }
    // f(index, logit) for every token of the row, each by one thread
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int s = threadIdx.x; s < n + 2; s += kRound * kT) {
            Slot u[kRound];
#pragma unroll
            for (int j = 0; j < kRound; ++j) u[j] = load(s + j * kT);
#pragma unroll
            for (int j = 0; j < kRound; ++j) {
                const int i = index(s + j * kT), end = s + j * kT == 0 ? head : V;
#pragma unroll
                for (int v = 0; v < kV; ++v)
                    if (i + v < end) f(i + v, u[j][v]);
            }
        }
    }
};

// --------------------------------------------------------------- sums

template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
    return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xF, false);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ uint64_t dpp_add(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, kCtrl, kRows, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), kCtrl, kRows, 0xF, false);
    return v + ((uint64_t)hi << 32 | lo);
}
// Sum of the lanes up to this one: shifts within rows of 16, then the last lane of a row to
// the next row, and of the lower half to the upper one.
template <class T>
__device__ __forceinline__ T wave_scan(T v) {
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    return dpp_add<0x143, 0xC>(v);
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (uint64_t)hi << 32 | lo;
}

struct Sums {
    uint64_t waves[2][kT / 64];
    uint64_t found[3];
    uint64_t one;
    int listed, matching;
};
struct Shared : Sums {
    union {
        uint64_t bins[kBins];
        ulonglong2 few[kFewest];  // place and weight
    };
    uint64_t list[kListed];
    uint64_t weights[kListed];
};

// Sum of the workgroup's values before this thread's, and of all.
__device__ __forceinline__ uint64_t scan(uint64_t v, Sums &sh, uint64_t &total) {
    const uint64_t s = wave_scan(v);
    lds_barrier();
    if ((threadIdx.x & 63) == 63) sh.waves[0][threadIdx.x >> 6] = s;
    lds_barrier();
    uint64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) {
        const uint64_t u = sh.waves[0][w];
        if (w < (int)(threadIdx.x >> 6)) before += u;
        total += u;
    }
    return before + s - v;
}
// Smallest of the wave's and of the workgroup's values (the moves of wave_scan; what a move does not
// reach keeps all ones).
template <int kCtrl, int kRows>
__device__ __forceinline__ uint64_t dpp_min(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(-1, (int)(uint32_t)v, kCtrl, kRows, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(-1, (int)(uint32_t)(v >> 32), kCtrl, kRows, 0xF, false);
    return min(v, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint64_t wave_smallest(uint64_t v) {
    v = dpp_min<0x111, 0xF>(v);
    v = dpp_min<0x112, 0xF>(v);
    v = dpp_min<0x114, 0xF>(v);
    v = dpp_min<0x118, 0xF>(v);
    v = dpp_min<0x142, 0xA>(v);
    return lane_value(dpp_min<0x143, 0xC>(v), 63);
}
__device__ __forceinline__ uint64_t smallest(uint64_t v, Sums &sh) {
    v = wave_smallest(v);
    lds_barrier();
    if ((threadIdx.x & 63) == 0) sh.waves[0][threadIdx.x >> 6] = v;
    lds_barrier();
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) v = min(v, sh.waves[0][w]);
    return v;
}

// The bin in which the running sum of the bins reaches limit(total), into sh.found: bin, sum before
// it, sum in it.  False where it does not.
template <class Limit>
__device__ __forceinline__ bool find_bin(const uint64_t (&bins)[kBins], Sums &sh, Limit limit, uint64_t &total, uint64_t &left) {
    constexpr int kEach = kBins / kT;
    uint64_t v[kEach], mine = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) mine += v[j] = bins[kEach * threadIdx.x + j];
    uint64_t before = scan(mine, sh, total);
    left = limit(total);
    if (left > total) return false;
    if (before < left && left <= before + mine) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (before < left && left <= before + v[j]) {
                sh.found[0] = kEach * threadIdx.x + j;
                sh.found[1] = before;
                sh.found[2] = v[j];
            }
            before += v[j];
        }
    }
    lds_barrier();
    return true;
}

// Adds a lane's weight to its bin; once for the wave where all add the same to one bin (rows of
// equal logits).
__device__ __forceinline__ void add_to(uint64_t *bins, int bin, uint64_t w) {
    const uint64_t active = __ballot(true);
    const uint64_t w0 = (uint64_t)__builtin_amdgcn_readfirstlane((int)(w >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)w);
    if (__ballot(bin == __builtin_amdgcn_readfirstlane(bin) && w == w0) != active) {
        atomicAdd((unsigned long long *)&bins[bin], (unsigned long long)w);
    } else if ((int)(threadIdx.x & 63) == __builtin_ctzll(active)) {
        atomicAdd((unsigned long long *)&bins[bin], (unsigned long long)(w0 * __builtin_popcountll(active)));
    }
}

// Where the running sum of `value` over the tokens, in the order of `order` (whole
// numbers of `bits` bits, no two the same), reaches limit(total): all ones where it
// does not.  Digit by digit: sums of the values by the next bits of the order, then the bin in
// which the running sum reaches the limit.  go(f) calls f(token) once for every token.
// `prefix`: the bits above them, the same for all.
// kLast: any number between that token's and the next one's will do.
// kFew: going through the tokens costs less than a digit; ends at a bin of one token.
template <bool kLast, bool kFew, class Go, class Order, class Value, class Limit>
__device__ __forceinline__ uint64_t reach(Shared &sh, int bits, uint64_t prefix, Go go, Order order, Value value, Limit limit,
                          uint64_t &total) {
    uint64_t left = 0;
    bool first = true;
    while (bits > 0) {
        const int digit = min(kDigit, bits), shift = bits - digit;
        for (int i = threadIdx.x; i < kBins; i += kT) sh.bins[i] = 0;
        if (threadIdx.x == 0) sh.matching = 0;
        lds_barrier();
        go([&](auto p) {
            const uint64_t o = order(p);
            if (!first && o >> bits != prefix) return;
            const uint64_t w = value(p);
            if (!w) return;
            const int bin = (int)(o >> shift) & ((1 << digit) - 1);
            if (kFew)
                atomicAdd((unsigned long long *)&sh.bins[bin], (unsigned long long)w);
            else
                add_to(sh.bins, bin, w);
        });
        lds_barrier();
        uint64_t sum;
        const uint64_t rest = left;
        const bool there = find_bin(sh.bins, sh, [&](uint64_t s) { return first ? limit(s) : rest; }, sum, left);
        if (first) total = sum;
        if (!there) return ~0ull;
        prefix = prefix << digit | sh.found[0];
        left -= sh.found[1];
        bits = shift;
        const bool whole = left == sh.found[2];  // the bin's last token
        if (kLast && whole) {
            lds_barrier();
            return ((prefix + 1) << shift) - 1;
        }
        if (kFew && bits > 0) {
            go([&](auto p) {
                const uint64_t o = order(p);
                if (o >> bits == prefix && value(p)) {
                    atomicAdd(&sh.matching, 1);
                    sh.one = o;
                }
            });
            lds_barrier();
            if (sh.matching == 1) {
                const uint64_t o = sh.one;
                lds_barrier();
                return o;
            }
        }
        lds_barrier();
        first = false;
    }
    return prefix;
}

// Of at most kFewest tokens (sh.few, filled up with all ones to a multiple of kBatch), a thread
// each: how many precede p in the order, and their weight.  (What is read from LDS grows with the square: 434
// tokens 12 us; 60 take 1.2, sorted 2.3.)
constexpr int kBatch = 8;
__device__ __forceinline__ int preceding(const Shared &sh, int n, uint64_t p, uint64_t &weight) {
    int rank = 0;
    weight = 0;
    for (int i = 0; i < n; i += kBatch) {
        ulonglong2 o[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) o[b] = sh.few[i + b];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const bool is = o[b].x < p;
            rank += is;
            weight += is ? o[b].y : 0;
        }
    }
    return rank;
}
// The sum of the workgroup's values.
__device__ __forceinline__ uint64_t sum_of(uint64_t v, Sums &sh) {
    uint64_t total;
    scan(v, sh, total);
    return total;
}

// The smaller (low) or the larger of a lane's value and that of the lane kApart from it (lane ^ kApart).
template <int kApart>
__device__ __forceinline__ uint64_t of_two(uint64_t x, bool low) {
    const uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
    uint64_t y;
    if constexpr (kApart == 32) {
        const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false), h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
        x = (uint64_t)h[0] << 32 | l[0];
        y = (uint64_t)h[1] << 32 | l[1];
    } else if constexpr (kApart == 16) {
        const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false), h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        x = (uint64_t)h[0] << 32 | l[0];
        y = (uint64_t)h[1] << 32 | l[1];
    } else {
        auto moved = [](uint32_t v) {
            constexpr int kCtrl = kApart == 8 ? 0x128 : kApart == 4 ? 0x141 : kApart == 2 ? 0x4E : 0xB1;
            v = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
            // (4: the lanes of 8 turned round, then those of 4)
            return kApart == 4 ? (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x1B, 0xF, 0xF, false) : v;
        };
        y = (uint64_t)moved(hi) << 32 | moved(lo);
    }
    return (x < y) == low ? x : y;
}
// Sorts the workgroup's numbers, of which the first n places (place i of x[0] in thread i, place kT + i of x[1])
// may hold others than all ones: bitonic, between lanes by moves of registers, further apart through
// sh.list.  (33 rows of 5003 tokens, k = 200: a call 21 us, with all compared with all 25.5; 8 bf16 rows with top-p
// 39 us and 45.5; through LDS alone the sort of 1024 took 9 us, digit by digit is faster.)
__device__ __forceinline__ void sort(uint64_t (&x)[2], int n, Shared &sh) {
    const int i = threadIdx.x;
    const bool two = n > kT;
    for (int level = 2; level / 2 < n; level *= 2) {
        const bool up[2] = {(i & level) == 0, ((i + kT) & level) == 0};
        auto each = [&](auto step) {
            x[0] = step(x[0], up[0]);
            if (two) x[1] = step(x[1], up[1]);
        };
        if (level == 2 * kT) {
            const uint64_t low = min(x[0], x[1]);
            x[1] = max(x[0], x[1]);
            x[0] = low;
        }
        for (int apart = min(level, kT) / 2; apart >= 64; apart /= 2) {
            sh.list[i] = x[0];
            if (two) sh.list[kT + i] = x[1];
            lds_barrier();
            const uint64_t y[2] = {sh.list[i ^ apart], two ? sh.list[kT + (i ^ apart)] : 0};
            lds_barrier();
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (e == 0 || two) x[e] = (x[e] < y[e]) == (((i & apart) == 0) == up[e]) ? x[e] : y[e];
        }
        if (__builtin_amdgcn_readfirstlane(i) >= 2 * n) continue;  // (a wave of no place of the next power of two)
        auto low = [&](int apart, bool up) { return ((i & apart) == 0) == up; };
        if (level >= 64) each([&](uint64_t v, bool up) { return of_two<32>(v, low(32, up)); });
        if (level >= 32) each([&](uint64_t v, bool up) { return of_two<16>(v, low(16, up)); });
        if (level >= 16) each([&](uint64_t v, bool up) { return of_two<8>(v, low(8, up)); });
        if (level >= 8) each([&](uint64_t v, bool up) { return of_two<4>(v, low(4, up)); });
        if (level >= 4) each([&](uint64_t v, bool up) { return of_two<2>(v, low(2, up)); });
        each([&](uint64_t v, bool up) { return of_two<1>(v, low(1, up)); });
    }
}

// --------------------------------------------------------------- part

// The sum of the waves' counts (one barrier; `turn` alternates).
__device__ __forceinline__ int block_count(int n, Sums &sh, int turn) {
    if ((threadIdx.x & 63) == 0) sh.waves[turn & 1][threadIdx.x >> 6] = n;
    lds_barrier();
    n = 0;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) n += (int)sh.waves[turn & 1][w];
    return n;
}
// How many of the workgroup's values are at least t.
template <int N>
__device__ __forceinline__ int count_from(const uint32_t (&v)[N], uint32_t t, Sums &sh, int turn) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) n += __builtin_popcountll(__ballot(v[j] >= t));
    return block_count(n, sh, turn);
}
// The largest t, bit by bit but for the last `low`, that at least k of the workgroup's values reach.
template <int N>
__device__ __forceinline__ uint32_t block_kth(const uint32_t (&v)[N], int k, int low, Sums &sh) {
    uint32_t t = 0;
    for (int bit = 31; bit >= low; --bit) {
        const int n = count_from(v, t | 1u << bit, sh, bit);
        if (n >= k) t |= 1u << bit;
        if (n == k) break;
    }
    return t;
}
// The same of a wave's values, but for the last ten bits.
template <int N>
__device__ __forceinline__ uint32_t wave_kth(const uint32_t (&v)[N], int k) {
    uint32_t t = 0;
    for (int bit = 31; bit >= 10; --bit) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) n += __builtin_popcountll(__ballot(v[j] >= (t | 1u << bit)));
        if (n >= k) t |= 1u << bit;
        if (n == k) break;
    }
    return t;
}

// Candidates: where k tokens are at least t, a token below t is not among the row's first k. A
// round of segments lists the tokens from t on.  t begins as the least of what each wave has an eighth
// of k vectors' largest tokens from (no barrier to find; k different tokens in all), and in a
// row of no special order hardly a token is listed after the first round.  Where the list
// gets full, t rises to the k-th largest of what is listed and of the new vectors' largest
// tokens.
template <bool kBF>
__global__ __launch_bounds__(kT) void sample_part_kernel(const Job j) {
    __shared__ struct : Sums {
        uint64_t list[kListed];
    } sh;
    using R = Row<kBF>;
    constexpr int kV = R::kV, kHeld = kListed / kT, kWaves = kT / 64;
    const int64_t r = blockIdx.x / j.parts;
    const int part = blockIdx.x % j.parts;
    const R row(j.a, r);
    const Limits lim(j.a, r);
    const bool lists = lim.listed();
    const int begin = (int)((int64_t)row.segments() * part / j.parts), end = (int)((int64_t)row.segments() * (part + 1) / j.parts);

    if (j.bins) {  // cleared for the next launch
        for (int i = part * kT + threadIdx.x; i < kBins; i += j.parts * kT) global(j.bins)[r * kBins + i] = 0;
        if (part == 0 && threadIdx.x == 0) j.steps[r] = 0;
    }
    if (threadIdx.x == 0) sh.listed = 0;

    float best = -INFINITY, from = -INFINITY;
    int best_slot = 0, listed = 0;
    bool full = false;  // uniform
    typename R::Slot u[kRound], next[kRound];
    auto load = [&](int s) {
#pragma unroll
        for (int n = 0; n < kRound; ++n) next[n] = row.load(s + n < end ? (s + n) * kT + threadIdx.x : row.n + 2);
    };
    load(begin);
    for (int s = begin; s < end; s += kRound) {
        float most[kRound];
        const int slot0 = s * kT + threadIdx.x;
#pragma unroll
        for (int n = 0; n < kRound; ++n) u[n] = next[n];
        if (s + kRound < end) load(s + kRound);
#pragma unroll
        for (int n = 0; n < kRound; ++n) {
            most[n] = u[n][0];
#pragma unroll
            for (int v = 1; v < kV; ++v) most[n] = fmaxf(most[n], u[n][v]);
            if (most[n] > best) {
                best = most[n];
                best_slot = slot0 + n * kT;
            }
        }
        if (!lists || full) continue;
        auto append = [&]() {
            // this lane's candidates as bits, then room for the wave's at once
            uint32_t mine = 0;
#pragma unroll
            for (int n = 0; n < kRound; ++n)
                if (__ballot(most[n] >= from))
#pragma unroll
                    for (int v = 0; v < kV; ++v)  // (-infinity is no candidate)
                        mine |= (uint32_t)(u[n][v] >= from && u[n][v] > -INFINITY) << (n * kV + v);
            if (__ballot(mine)) {
                const uint32_t upto = wave_scan((uint32_t)__builtin_popcount(mine));
                int at = 0;
                if ((threadIdx.x & 63) == 63) at = atomicAdd(&sh.listed, (int)upto);
                at = __builtin_amdgcn_readlane(at, 63) + (int)upto - __builtin_popcount(mine);
#pragma unroll
                for (int n = 0; n < kRound; ++n) {
                    const uint32_t here = mine >> (n * kV) & ((1u << kV) - 1);
                    if (!__ballot(here)) continue;
#pragma unroll
                    for (int v = 0; v < kV; ++v) {
                        if (!(here >> v & 1)) continue;
                        if (at < kListed) sh.list[at] = place(order_key(u[n][v]), row.index(slot0 + n * kT) + v);
                        ++at;
                    }
                }
            }
            lds_barrier();
            const int n = sh.listed;
            lds_barrier();
            return n;
        };
        if (s == begin) {
            uint32_t w[kRound];
#pragma unroll
            for (int n = 0; n < kRound; ++n) w[n] = order_key(most[n]);
            const uint32_t t = wave_kth(w, (lim.k + kWaves - 1) / kWaves);
            if ((threadIdx.x & 63) == 0) sh.waves[0][threadIdx.x >> 6] = t;
            lds_barrier();
            uint32_t least = ~0u;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) least = min(least, (uint32_t)sh.waves[0][w]);
            if (least <= kNothing) {  // a wave at the row's end has fewer
                lds_barrier();
                least = block_kth(w, lim.k, 10, sh);
            }
            if (least > kNothing) from = key_value(least);
        }
        int now = append();
        if (now > kListed) {
            // the k-th largest of the listed tokens and the new vectors' largest
            uint64_t held[kHeld];
            uint32_t w[kHeld + kRound];
#pragma unroll
            for (int n = 0; n < kHeld; ++n) {
                const int i = n * kT + threadIdx.x;
                held[n] = i < listed ? sh.list[i] : ~0ull;
                w[n] = i < listed ? place_key(held[n]) : 0;
            }
#pragma unroll
            for (int n = 0; n < kRound; ++n) w[kHeld + n] = order_key(most[n]);
            uint32_t t = block_kth(w, lim.k, 0, sh);
            if (t <= kNothing) {  // fewer vectors than k: the k-th largest of the new tokens themselves
                t = 0;
                for (int bit = 31; bit >= 0; --bit) {
                    const float f = key_value(t | 1u << bit);
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < kRound; ++i)
#pragma unroll
                        for (int v = 0; v < kV; ++v) n += __builtin_popcountll(__ballot(u[i][v] >= f));
                    if (block_count(n, sh, bit) >= lim.k) t |= 1u << bit;
                }
            }
            from = t > kNothing ? fmaxf(from, key_value(t)) : from;
            if (threadIdx.x == 0) sh.listed = 0;
            lds_barrier();
#pragma unroll
            for (int n = 0; n < kHeld; ++n)
                if (held[n] != ~0ull && place_key(held[n]) >= order_key(from)) sh.list[atomicAdd(&sh.listed, 1)] = held[n];
            lds_barrier();
            now = append();
            full = now > kListed;
        }
        listed = now;
    }
    // the first of the largest tokens: each thread's largest vector again
    uint64_t first = ~0ull;
    const uint32_t key = order_key(best);
    const uint32_t top = place_key(smallest(place(key, 0), sh));
    if (key == top && top > kNothing) {
        const typename R::Slot u = row.load(best_slot);
#pragma unroll
        for (int v = kV - 1; v >= 0; --v)
            if (order_key(u[v]) == top) first = place(top, row.index(best_slot) + v);
    }
    first = smallest(first, sh);
    if (threadIdx.x == 0) {
        global(j.first)[r * j.parts + part] = first;
        if (lists) global(j.counts)[r * j.parts + part] = full ? kTooMany : listed;
    }
    if (lists) {
        const int size = kT / j.groups;
        float top = best;
        for (int o = 1; o < size; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        if (threadIdx.x % size == 0) global(j.tops)[(r * j.parts + part) * j.groups + threadIdx.x / size] = order_key(top);
    }
    if (lists && !full) {
        const auto list = global(j.lists) + (r * j.parts + part) * kListed;
        for (int i = threadIdx.x; i < listed; i += kT) list[i] = sh.list[i];
    }
}

// The first place of a row (all ones: no token can be drawn), in every wave by itself.
__device__ __forceinline__ uint64_t first_place(const Job &j, int64_t r) {
    uint64_t first = ~0ull;
    for (int p = threadIdx.x & 63; p < j.parts; p += 64) first = min(first, global(j.first)[r * j.parts + p]);
    return wave_smallest(first);
}

// --------------------------------------------------------------- bins and step

template <bool kBF>
__global__ __launch_bounds__(kT) void sample_bins_kernel(const Job j) {
    __shared__ uint64_t bins[kBins];
    using R = Row<kBF>;
    const int64_t r = blockIdx.x / j.cuts;
    const int part = blockIdx.x % j.cuts;
    const R row(j.a, r);
    const Limits lim(j.a, r);
    const int begin = (int)((int64_t)row.segments() * part / j.cuts), end = (int)((int64_t)row.segments() * (part + 1) / j.cuts);
    typename R::Slot u[kRound], next[kRound];
    auto load = [&](int s) {
#pragma unroll
        for (int n = 0; n < kRound; ++n) next[n] = row.load(s + n < end ? (s + n) * kT + threadIdx.x : row.n + 2);
    };
    load(begin);  // on its way while the rest of the row's state is read
    const uint64_t first = first_place(j, r);
    if (!lim.binned() || !(lim.top_p < 1.0f) || first == ~0ull) return;
    const Weights weight(place_key(first), lim);
    const float cut = weight.cut(kBins);
    for (int i = threadIdx.x; i < kBins; i += kT) bins[i] = 0;
    __syncthreads();
    for (int s = begin; s < end; s += kRound) {
#pragma unroll
        for (int n = 0; n < kRound; ++n) u[n] = next[n];
        if (s + kRound < end) load(s + kRound);
#pragma unroll
        for (int n = 0; n < kRound; ++n) {
            if (s + n >= end) break;
#pragma unroll
            for (int v = 0; v < R::kV; ++v) {
                const float l = u[n][v];
                if (!(l >= cut)) continue;
                double x;
                const int b = weight.bin(l, x);
                const uint64_t w = weight.at(l, x);
                if (w) atomicAdd((unsigned long long *)&bins[b], (unsigned long long)w);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kT)
        if (bins[i]) atomicAdd((unsigned long long *)&j.bins[r * kBins + i], (unsigned long long)bins[i]);
}

constexpr int kStepHere = 1024;  // tokens of the step that a workgroup gathers in LDS

template <bool kBF>
__global__ __launch_bounds__(kT) void sample_step_kernel(const Job j) {
    __shared__ struct : Sums {
        uint64_t bins[kBins], sums[kRound][kT / 64], step[kStepHere];
    } sh;
    using R = Row<kBF>;
    const int64_t r = blockIdx.x / j.cuts;
    const int part = blockIdx.x % j.cuts;
    const R row(j.a, r);
    const Limits lim(j.a, r);
    const int begin = (int)((int64_t)row.segments() * part / j.cuts), end = (int)((int64_t)row.segments() * (part + 1) / j.cuts);
    typename R::Slot u[kRound], next[kRound];
    auto load = [&](int s) {
#pragma unroll
        for (int n = 0; n < kRound; ++n) next[n] = row.load(s + n < end ? (s + n) * kT + threadIdx.x : row.n + 2);
    };
    load(begin);  // on its way while the rest of the row's state is read
    const uint64_t first = first_place(j, r);
    if (!lim.binned() || first == ~0ull) return;
    const Weights weight(place_key(first), lim);
    const uint64_t least = lim.least();
    int last = kBins;  // the step in which top-p ends
    if (threadIdx.x == 0) sh.listed = 0;
    if (lim.top_p < 1.0f) {
        for (int i = threadIdx.x; i < kBins; i += kT) sh.bins[i] = global(j.bins)[r * kBins + i];
        __syncthreads();
        uint64_t total, left;
        if (find_bin(sh.bins, sh, [&](uint64_t s) { return lim.end(s); }, total, left)) {
            last = (int)sh.found[0];
            if (part == 0 && threadIdx.x == 0) global(j.ends)[2 * r + 1] = left - sh.found[1];
        }
    }
    if (part == 0 && threadIdx.x == 0) global(j.ends)[2 * r] = last;
    const float cut = weight.cut(last);
    for (int s = begin; s < end; s += kRound) {
#pragma unroll
        for (int n = 0; n < kRound; ++n) u[n] = next[n];
        if (s + kRound < end) load(s + kRound);
        uint64_t sum[kRound];
#pragma unroll
        for (int n = 0; n < kRound; ++n) {
            sum[n] = 0;
            if (s + n >= end) break;
#pragma unroll
            for (int v = 0; v < R::kV; ++v) {
                const float l = u[n][v];
                if (!(l >= cut)) continue;
                double x;
                const int b = weight.bin(l, x);
                if (b > last) continue;
                if (b == last) {
                    const uint64_t p = place(order_key(l), row.index((s + n) * kT + threadIdx.x) + v);
                    const int here = atomicAdd(&sh.listed, 1);
                    if (here < kStepHere) {
                        sh.step[here] = p;
                    } else {
                        const uint32_t at = atomicAdd(&j.steps[r], 1u);
                        if (at < kListed) global(j.step)[r * kListed + at] = p;
                    }
                } else {
                    const uint64_t w = weight.at(l, x);
                    if (w >= least) sum[n] += w;
                }
            }
            sum[n] = lane_value(wave_scan(sum[n]), 63);
        }
        // the segments' sums, one barrier pair for the round
        lds_barrier();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < kRound; ++n) sh.sums[n][threadIdx.x >> 6] = sum[n];
        lds_barrier();
        if (threadIdx.x < kRound && s + (int)threadIdx.x < end) {
            uint64_t all = 0;
#pragma unroll
            for (int w = 0; w < kT / 64; ++w) all += sh.sums[threadIdx.x][w];
            global(j.sums)[r * j.segments + s + threadIdx.x] = all;
        }
    }
    __syncthreads();
    const int here = min(sh.listed, kStepHere);
    if (here == 0) return;
    if (threadIdx.x == 0) sh.matching = (int)atomicAdd(&j.steps[r], (uint32_t)here);
    __syncthreads();
    for (int i = threadIdx.x; i < here; i += kT)
        if ((uint32_t)sh.matching + i < kListed) global(j.step)[r * kListed + sh.matching + i] = sh.step[i];
}

// --------------------------------------------------------------- row

// The index at which the running sum of kept weights is over min(floor(u sum), sum - 1).
__device__ __forceinline__ uint64_t target(float u, uint64_t sum) {
    return 1 + min((uint64_t)((double)fmaxf(u, 0.0f) * (double)sum), sum - 1);
}

template <bool kBF>
__global__ __launch_bounds__(kT) void sample_row_kernel(const Job j) {
    __shared__ Shared sh;
    using R = Row<kBF>;
    const s3d8_sample_args &a = j.a;
    const int64_t r = blockIdx.x;
    const R row(a, r);
    Limits lim(a, r);
    // (asked for before any of it is used)
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tops = j.parts * j.groups;
    const int64_t at0 = r * j.parts;
    uint32_t count = 0, some[256 / 64] = {};
    if (!j.direct && j.counts && lim.listed()) {
        if (lane < j.parts) count = global(j.counts)[at0 + lane];
        if (wave == 0 && tops <= 256)
#pragma unroll
            for (int i = 0; i < 256 / 64; ++i)
                if (i * 64 + lane < tops) some[i] = global(j.tops)[at0 * j.groups + i * 64 + lane];
    }
    uint64_t first;
    int n = 0, bits = 0;  // tokens in sh.list, bits in which their places differ
    if (j.direct) {  // all tokens of the row
        constexpr int kMine = kListed / kT;
        float l[kMine];
#pragma unroll
        for (int q = 0; q < kMine; ++q) l[q] = row.one(min(q * kT + (int)threadIdx.x, row.V - 1));
        first = ~0ull;
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int i = q * kT + threadIdx.x;
            if (i >= row.V) break;
            const uint32_t key = order_key(l[q]);
            sh.list[i] = place(key, i);
            if (key > kNothing) first = min(first, sh.list[i]);
        }
        first = smallest(first, sh);
        n = row.V;
        bits = kOrderBits;
        if (lim.k == 0) lim.k = kListed;
    } else {
        first = first_place(j, r);
    }
    if (first == ~0ull || lim.greedy) {
        if (threadIdx.x == 0) {
            global(a.token)[r] = first == ~0ull ? -1 : (int32_t)place_index(first);
            if (a.prob) global(a.prob)[r] = first == ~0ull ? 0.0f : 1.0f;
        }
        return;
    }
    const Weights weight(place_key(first), lim);
    const uint64_t least = lim.least();
    const float u = global(a.u)[r];
    auto answer = [&](uint32_t token, uint64_t w, uint64_t total) {
        global(a.token)[r] = (int32_t)token;
        if (a.prob) global(a.prob)[r] = (float)((double)w / (double)total);
    };
    auto by_place = [](uint64_t p) { return p; };
    uint64_t total;

    bool fits = j.direct;
    if (!j.direct && lim.listed()) {
        // `from`: the k-th largest of the parts' tops, as k tokens are at least that (0: too few
        // tops). What the parts listed from there on: each wave takes some parts' lists, two
        // loads a lane of four lists on their way at once.
        uint32_t from = 0;
        fits = !__ballot(count == kTooMany);
        constexpr int kWaves = kT / 64;
        if (tops > 256) {
            uint32_t w[kTops / kT];
#pragma unroll
            for (int i = 0; i < kTops / kT; ++i)
                w[i] = i * kT + (int)threadIdx.x < tops ? global(j.tops)[at0 * j.groups + i * kT + threadIdx.x] : 0;
            from = block_kth(w, lim.k, 10, sh);
        } else {
            if (wave == 0) {
                from = wave_kth(some, lim.k);
                if (lane == 0) sh.one = from;
            }
            lds_barrier();
            from = (uint32_t)sh.one;
        }
        if (threadIdx.x == 0) sh.listed = 0;
        lds_barrier();
        if (fits) {
            // the lists in pieces of 64 tokens, piece by piece of each part in turn: four of a wave's are
            // on their way at once
            constexpr int kAhead = 4;
            uint32_t longest = count;
#pragma unroll
            for (int o = 1; o < kMaxParts; o <<= 1) longest = max(longest, (uint32_t)__shfl_xor((int)longest, o));
            const int pieces = (int)(__builtin_amdgcn_readfirstlane((int)longest) + 63) / 64 * j.parts;
            for (int q = wave; q < pieces; q += kAhead * kWaves) {
                uint64_t x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int piece = q + i * kWaves, p = piece % j.parts, at = piece / j.parts * 64 + lane;
                    x[i] = at < __builtin_amdgcn_readlane((int)count, p) ? global(j.lists)[(at0 + p) * kListed + at] : ~0ull;
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const bool in = x[i] != ~0ull && place_key(x[i]) >= from;
                    if (!__ballot(in)) continue;
                    if (in) {
                        const int at = atomicAdd(&sh.listed, 1);
                        if (at < kListed) sh.list[at] = x[i];
                        if (x[i] != first) bits = max(bits, 64 - __builtin_clzll(x[i] ^ first));
                    }
                }
            }
        }
        lds_barrier();
        n = sh.listed;
        if (fits && n > kListed) {  // the k-th place by the lists themselves
            auto go = [&](auto f) {
                for (int p = wave; p < j.parts; p += kWaves)
                    for (int i = lane; i < (int)global(j.counts)[at0 + p]; i += 64) f(global(j.lists)[(at0 + p) * kListed + i]);
            };
            const uint64_t last = reach<true, false>(
                sh, kOrderBits, 0, go, by_place, [](uint64_t) { return 1ull; }, [&](uint64_t) { return (uint64_t)lim.k; }, total);
            if (threadIdx.x == 0) sh.listed = 0;
            lds_barrier();
            bits = kOrderBits;
            go([&](uint64_t x) {
                if (x <= last) sh.list[atomicAdd(&sh.listed, 1)] = x;
            });
            lds_barrier();
            n = sh.listed;
        }
    }
    if (fits && n <= kFewest) {
        // fewest: each thread compares its token with all of them, by place for what is kept, then by index
        uint64_t p = ~0ull, w = 0;
        if ((int)threadIdx.x < n) {
            p = sh.list[threadIdx.x];
            w = weight(place_key(p));
        }
        int at = (int)threadIdx.x < n ? (int)threadIdx.x : -1;
        for (int pass = 0; pass < 2; ++pass) {
            if (at >= 0) sh.few[at] = make_ulonglong2(p, w);
            if (threadIdx.x < kBatch - 1 && n + threadIdx.x < kFewest) sh.few[n + threadIdx.x] = make_ulonglong2(~0ull, 0);
            if (pass) total = sum_of(w, sh);
            lds_barrier();
            uint64_t before = 0;
            const int rank = at >= 0 ? preceding(sh, n, p, before) : kListed;
            if (pass) {
                const uint64_t left = target(u, total);
                if (at >= 0 && before < left && left <= before + w) answer((uint32_t)p, w, total);
                return;
            }
            bool kept = rank < lim.k;
            if (lim.top_p < 1.0f) {
                const uint64_t sum = sum_of(kept ? w : 0, sh);
                kept = kept && before < lim.end(sum);
            }
            if (!kept || w < least) w = 0;
            p = place_index(p);
            if (threadIdx.x == 0) sh.listed = 0;
            lds_barrier();
            at = w ? atomicAdd(&sh.listed, 1) : -1;
            lds_barrier();
            n = sh.listed;
        }
    }
    // those of the list at this thread's places
    auto listed = [&](uint64_t(&x)[2], int n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = e * kT + (int)threadIdx.x < n ? sh.list[e * kT + threadIdx.x] : ~0ull;
    };
    // the weights of the first `most` of n sorted tokens, and the sums before them
    auto weigh = [&](const uint64_t(&x)[2], int n, int most, bool by_index, uint64_t(&w)[2], uint64_t(&before)[2]) {
        total = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            w[e] = before[e] = 0;
            if (e * kT >= n) break;
            if (e * kT + (int)threadIdx.x < most) w[e] = weight(by_index ? (uint32_t)x[e] : place_key(x[e]));
            uint64_t sum;
            before[e] = total + scan(w[e], sh, sum);
            total += sum;
        }
    };
    if (fits && n <= kFewTokens) {
        // few: sorted by place for what is kept, the first of them, then by index
        uint64_t x[2], w[2], before[2];
        listed(x, n);
        for (int pass = 0; pass < 2; ++pass) {
            sort(x, n, sh);
            weigh(x, n, pass ? n : min(n, lim.k), pass, w, before);
            const uint64_t left = pass ? target(u, total) : lim.top_p < 1.0f ? lim.end(total) : ~0ull;
            uint64_t out = kFewTokens;  // the first place that is not kept
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (pass) {
                    if (before[e] < left && left <= before[e] + w[e]) answer((uint32_t)(x[e] >> 32), w[e], total);
                } else if (w[e] && w[e] >= least && before[e] < left) {
                    x[e] = (uint64_t)place_index(x[e]) << 32 | place_key(x[e]);
                } else {
                    x[e] = ~0ull;
                    out = min(out, (uint64_t)(e * kT + threadIdx.x));
                }
            }
            if (pass) return;
            n = (int)smallest(out, sh);
        }
    }
    if (fits) {
        bits = kOrderBits - (int)smallest((uint64_t)(kOrderBits - bits), sh);
        // top-k, top-p, the token: one piece of code, so that it is fetched once
        uint64_t end = ~0ull;
        for (int stage = 0; stage < 3; ++stage) {
            if (stage == 0 ? n <= lim.k : stage == 1 && !(lim.top_p < 1.0f)) {
                if (stage == 0) lds_barrier();
            } else {
                const uint64_t found = reach<false, true>(
                    sh, stage == 2 ? kIndexBits : bits, stage == 2 ? 0 : first >> bits,
                    [&](auto f) {
                        for (int i = threadIdx.x; i < n; i += kT) f(i);
                    },
                    [&](int i) { return stage == 2 ? place_index(sh.list[i]) : sh.list[i]; },
                    [&](int i) -> uint64_t {
                        if (stage == 0) return 1;
                        const uint64_t w = sh.weights[i];
                        return stage == 1 || (sh.list[i] <= end && w >= least) ? w : 0;
                    },
                    [&](uint64_t s) { return stage == 0 ? (uint64_t)lim.k : stage == 1 ? lim.end(s) : target(u, s); },
                    total);
                if (stage == 2) {
                    for (int i = threadIdx.x; i < n; i += kT)
                        if (place_index(sh.list[i]) == found) answer((uint32_t)found, sh.weights[i], total);
                    return;
                }
                end = found;
            }
            if (stage == 0) {  // those kept, with their weights
                uint64_t held[kListed / kT];
#pragma unroll
                for (int i = 0; i < kListed / kT; ++i) {
                    const int at = i * kT + threadIdx.x;
                    held[i] = at < n ? sh.list[at] : ~0ull;
                }
                if (threadIdx.x == 0) sh.listed = 0;
                lds_barrier();
#pragma unroll
                for (int i = 0; i < kListed / kT; ++i)
                    if (held[i] != ~0ull && held[i] <= end) {
                        const int at = atomicAdd(&sh.listed, 1);
                        sh.list[at] = held[i];
                        sh.weights[at] = weight(place_key(held[i]));
                    }
                lds_barrier();
                n = sh.listed;
                end = ~0ull;
            }
        }
    }
    if (!j.direct && lim.binned()) {
        const int last = (int)global(j.ends)[2 * r];
        const uint32_t n = last < kBins ? j.steps[r] : 0;
        if (n <= kListed) {
            // the exact end of top-p in its step
            for (int i = threadIdx.x; i < (int)n; i += kT) sh.list[i] = global(j.step)[r * kListed + i];
            __syncthreads();
            auto go = [&](auto f) {
                for (int i = threadIdx.x; i < (int)n; i += kT) f(sh.list[i]);
            };
            uint64_t end = ~0ull;
            if (n && n <= kFewTokens) {
                const uint64_t left = global(j.ends)[2 * r + 1];
                uint64_t x[2], w[2], before[2];
                listed(x, n);
                sort(x, n, sh);
                weigh(x, n, n, false, w, before);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (before[e] < left && left <= before[e] + w[e]) sh.one = x[e];
                    if (e * kT + threadIdx.x < n) sh.list[e * kT + threadIdx.x] = x[e];
                }
                __syncthreads();
                end = sh.one;
            } else if (n) {
                int bits = 0;
                const uint64_t some = sh.list[0];
                go([&](uint64_t p) { bits = p == some ? bits : max(bits, 64 - __builtin_clzll(p ^ some)); });
                bits = kOrderBits - (int)smallest((uint64_t)(kOrderBits - bits), sh);
                end = reach<true, true>(
                    sh, bits, some >> bits, go, by_place, [&](uint64_t p) { return weight(place_key(p)); },
                    [&](uint64_t) { return global(j.ends)[2 * r + 1]; }, total);
            }
            // the segments' sums with it, and the segment of the random number
            const int segments = row.segments();
            for (int i = threadIdx.x; i < kBins; i += kT) sh.bins[i] = i < segments ? global(j.sums)[r * j.segments + i] : 0;
            __syncthreads();
            go([&](uint64_t p) {
                const uint64_t w = p <= end ? weight(place_key(p)) : 0;
                if (w && w >= least)
                    atomicAdd((unsigned long long *)&sh.bins[row.slot(place_index(p)) / kT], (unsigned long long)w);
            });
            __syncthreads();
            uint64_t left;
            find_bin(sh.bins, sh, [&](uint64_t s) { return target(u, s); }, total, left);
            left -= sh.found[1];
            const int slot = (int)sh.found[0] * kT + threadIdx.x;
            const typename R::Slot v = row.load(slot);
            uint64_t w[R::kV], mine = 0;
#pragma unroll
            for (int i = 0; i < R::kV; ++i) {
                double x;
                const int b = weight.bin(v[i], x);
                const bool in = b < last || (b == last && place(order_key(v[i]), row.index(slot) + i) <= end);
                w[i] = in ? weight.at(v[i], x) : 0;
                if (w[i] < least) w[i] = 0;
                mine += w[i];
            }
            uint64_t all, before = scan(mine, sh, all);
            if (before < left && left <= before + mine)
#pragma unroll
                for (int i = 0; i < R::kV; ++i) {
                    if (before < left && left <= before + w[i]) answer(row.index(slot) + i, w[i], total);
                    before += w[i];
                }
            return;
        }
    }

    // any row: digit by digit
    auto go = [&](auto f) { row.each([&](int i, float l) { f(place(order_key(l), i)); }); };
    uint64_t last = ~0ull;
    if (lim.k > 0)
        last = reach<true, false>(
            sh, kOrderBits, 0, go, by_place, [](uint64_t) { return 1ull; }, [&](uint64_t) { return (uint64_t)lim.k; }, total);
    auto ranked = [&](uint64_t p) { return p <= last ? weight(place_key(p)) : 0ull; };
    if (lim.top_p < 1.0f) {
        const uint64_t end = reach<true, false>(
            sh, kOrderBits, 0, go, by_place, ranked, [&](uint64_t s) { return lim.end(s); }, total);
        last = min(last, end);
    }
    const uint64_t index = reach<false, false>(
        sh, kIndexBits, 0, go, [](uint64_t p) { return (uint64_t)place_index(p); },
        [&](uint64_t p) {
            const uint64_t w = ranked(p);
            return w >= least ? w : 0ull;
        },
        [&](uint64_t s) { return target(u, s); }, total);
    if (threadIdx.x == 0) answer((uint32_t)index, weight(order_key(row.one((int)index))), total);
}

// --------------------------------------------------------------- host

struct Plan {
    int64_t rows, parts, cuts, segments, groups;
    bool direct, lists, bins, top_p;
    int64_t first, counts, lists_at, tops, bins_at, step, sums, ends, steps, bytes;
};

// As many parts as fill the device twice over, of at least a round of segments.
Plan plan(const s3d8_sample_args &a, int cus) {
    Plan p{};
    p.rows = std::min(a.M, kRowsAtOnce);
    const int64_t vectors = a.V / (a.type == S3D8_ROWS_BF16 ? 8 : 4) + 2;
    p.segments = (vectors + kT - 1) / kT;
    const bool one_k = !a.top_k, k_on = a.top_k_all > 0 && a.top_k_all < a.V;
    // Parts: of kRound segments at least, so that all of a thread's loads are on their way at once; four
    // workgroups for every CU (eight: 47 us for 40 with 128 rows, k = 50); and at least 16 k tokens, as the
    // candidates are the fewer the larger a part is beside k (k = 1000 of one row: 101 us in 32 parts, 50 in 8).
    const int64_t most = !one_k || !k_on ? kMaxParts : std::max<int64_t>(4, a.V / (16 * (int64_t)a.top_k_all));
    p.parts = std::max<int64_t>(1, std::min<int64_t>({(p.segments + kRound - 1) / kRound, 4 * cus / p.rows, kMaxParts, most}));
    // (the launches that take every weight have work for smaller parts: a segment at least)
    p.cuts = std::max<int64_t>(1, std::min<int64_t>(p.segments, 4 * cus / p.rows));
    // (V = 19 to 3500: 17 to 29 us, through the parts 15 to 45)
    p.direct = a.V <= kListed;
    p.lists = !one_k || (k_on && a.top_k_all <= kMaxTopK);
    p.bins = !one_k || !k_on;
    // four times as many tops as tokens that are kept, so that hardly more than those are at least the k-th of them
    const int64_t tops = !one_k || a.top_k_all > 256 ? kTops : a.top_k_all > 64 ? kTops / 4 : 256;
    static_assert(kMaxParts * 8 <= 256, "");
    for (p.groups = 256; p.groups > 8 && p.groups * p.parts > tops;) p.groups /= 2;
    p.top_p = a.top_p || a.top_p_all < 1.0f;
    if (p.direct) return p;
    int64_t at = 0;
    auto room = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 15) / 16 * 16;
        return here;
    };
    p.first = room(p.rows * p.parts * 8);
    p.counts = room(p.lists ? p.rows * p.parts * 4 : 0);
    p.lists_at = room(p.lists ? p.rows * p.parts * kListed * 8 : 0);
    p.tops = room(p.lists ? p.rows * p.parts * p.groups * 4 : 0);
    p.bins_at = room(p.bins ? p.rows * kBins * 8 : 0);
    p.step = room(p.bins ? p.rows * kListed * 8 : 0);
    p.sums = room(p.bins ? p.rows * p.segments * 8 : 0);
    p.ends = room(p.bins ? p.rows * 16 : 0);
    p.steps = room(p.bins ? p.rows * 4 : 0);
    p.bytes = at;
    return p;
}

int check_sizes(const s3d8_sample_args &a) {
    if (a.M <= 0 || a.V <= 0) return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (a.V > kMaxVocabulary) return s3d8::fail(S3D8_ERR_SHAPE, "more than 262144 tokens are not supported");
    if (a.M > kMaxRows) return s3d8::fail(S3D8_ERR_SHAPE, "more than 524288 rows are not supported");
    if (a.type != S3D8_ROWS_F32 && a.type != S3D8_ROWS_BF16) return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    return S3D8_OK;
}

template <bool kBF>
void launch(const Job &j, const Plan &p, int64_t rows, hipStream_t stream) {
    const dim3 each((unsigned)(rows * p.parts)), cut((unsigned)(rows * p.cuts)), threads(kT);
    if (!p.direct) hipLaunchKernelGGL(sample_part_kernel<kBF>, each, threads, 0, stream, j);
    if (!p.direct && p.bins && p.top_p) hipLaunchKernelGGL(sample_bins_kernel<kBF>, cut, threads, 0, stream, j);
    if (!p.direct && p.bins) hipLaunchKernelGGL(sample_step_kernel<kBF>, cut, threads, 0, stream, j);
    hipLaunchKernelGGL(sample_row_kernel<kBF>, dim3((unsigned)rows), threads, 0, stream, j);
}

}  // namespace

extern "C" {

int64_t s3d8_sample_workspace_bytes(const s3d8_sample_args *args, int32_t num_cus) {
    if (!args || num_cus <= 0 || check_sizes(*args)) return -1;
    s3d8::clear_error();
    return plan(*args, num_cus).bytes;
}

int32_t s3d8_sample(const s3d8_sample_args *args, void *stream) {
    if (!args || !args->logits || !args->u || !args->token) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    const s3d8_sample_args &a = *args;
    int rc = check_sizes(a);
    if (rc) return rc;
    if ((a.M > 1 && a.row < a.V) || a.row < 0 || a.row > int64_t(1) << 40)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "rows must be at least V elements apart (and at most 2^40)");
    if (!a.temperature && !(a.temperature_all >= 0.0f && a.temperature_all <= 0x1p100f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "temperature must be from 0 to 2^100");
    if (!a.top_k && a.top_k_all < 0) return s3d8::fail(S3D8_ERR_INVALID_ARG, "top_k must not be negative");
    if (!a.top_p && !(a.top_p_all >= 0.0f && a.top_p_all <= 1.0f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "top_p must be from 0 to 1");
    if (!a.min_p && !(a.min_p_all >= 0.0f && a.min_p_all <= 1.0f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "min_p must be from 0 to 1");
    auto odd = [](const void *p, uintptr_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; };
    if (odd(a.logits, a.type == S3D8_ROWS_F32 ? 4 : 2) || odd(a.u, 4) || odd(a.temperature, 4) || odd(a.top_k, 4) ||
        odd(a.top_p, 4) || odd(a.min_p, 4) || odd(a.token, 4) || odd(a.prob, 4) || odd(a.workspace, 16))
        return s3d8::fail(S3D8_ERR_ALIGN, "arrays must be aligned to an element, the workspace to 16 bytes");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    const Plan p = plan(a, cus);
    if (p.bytes > 0 && (!a.workspace || a.workspace_bytes < p.bytes))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "workspace smaller than s3d8_sample_workspace_bytes");
    char *const ws = static_cast<char *>(a.workspace);
    for (int64_t r = 0; r < a.M; r += p.rows) {
        Job j{};
        j.a = a;
        j.a.logits = static_cast<const char *>(a.logits) + r * a.row * (a.type == S3D8_ROWS_F32 ? 4 : 2);
        j.a.u += r;
        if (a.temperature) j.a.temperature += r;
        if (a.top_k) j.a.top_k += r;
        if (a.top_p) j.a.top_p += r;
        if (a.min_p) j.a.min_p += r;
        j.a.token += r;
        if (a.prob) j.a.prob += r;
        j.direct = p.direct;
        j.parts = (int)p.parts;
        j.cuts = (int)p.cuts;
        j.segments = (int)p.segments;
        j.first = reinterpret_cast<uint64_t *>(ws + p.first);
        j.counts = p.lists ? reinterpret_cast<uint32_t *>(ws + p.counts) : nullptr;
        j.lists = reinterpret_cast<uint64_t *>(ws + p.lists_at);
        j.tops = reinterpret_cast<uint32_t *>(ws + p.tops);
        j.groups = (int)p.groups;
        j.bins = p.bins ? reinterpret_cast<uint64_t *>(ws + p.bins_at) : nullptr;
        j.step = reinterpret_cast<uint64_t *>(ws + p.step);
        j.sums = reinterpret_cast<uint64_t *>(ws + p.sums);
        j.ends = reinterpret_cast<uint64_t *>(ws + p.ends);
        j.steps = reinterpret_cast<uint32_t *>(ws + p.steps);
        const int64_t rows = std::min(p.rows, a.M - r);
        if (a.type == S3D8_ROWS_BF16)
            launch<true>(j, p, rows, (hipStream_t)stream);
        else
            launch<false>(j, p, rows, (hipStream_t)stream);
    }
    return s3d8::launch_status();
}

}  // extern "C"
