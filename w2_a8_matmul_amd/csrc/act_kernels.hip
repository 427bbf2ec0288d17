// What stands between the linear layers of a block, for gfx950: the norms
// before and after it with its gate and the residual sum, and the gated
// activation, each ending in the INT8 codes that the linear kernels read.
//
// Both are bound by memory: a row is read once, stays in the registers of one
// workgroup through its reductions, and is written once.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

constexpr int64_t kMaxWidth = 65536;    // 16 float4 per thread of 1024
constexpr int64_t kMaxRows = 1 << 19;   // keeps a launch under 2^32 threads

__device__ __forceinline__ float4 bf16x4_values(uint2 u) {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// A workgroup's share of a row of K fp32 or bf16 values from element `base`: thread
// t of T takes float4 t, t + T, ... (zeros past the row).
template <int T, int NV>
__device__ __forceinline__ void load_row(float4 (&v)[NV], const void *p, int64_t base, int n4, bool bf) {
    if (bf) {
        uint2 u[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * T;
            u[j] = i < n4 ? reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + base)[i] : make_uint2(0, 0);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = bf16x4_values(u[j]);
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * T;
            v[j] = i < n4 ? reinterpret_cast<const float4 *>(static_cast<const float *>(p) + base)[i]
                          : make_float4(0, 0, 0, 0);
        }
    }
}

__device__ __forceinline__ uint2 bf16x4(float4 v) {
    return make_uint2(f32_to_bf16_rne(v.x) | (uint32_t)f32_to_bf16_rne(v.y) << 16,
                      f32_to_bf16_rne(v.z) | (uint32_t)f32_to_bf16_rne(v.w) << 16);
}

__device__ __forceinline__ void store4(void *p, int64_t at, float4 v, bool bf) {
    if (bf)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at) = bf16x4(v);
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) = v;
}

template <class F>
__device__ __forceinline__ float4 map4(float4 a, F f) {
    return make_float4(f(a.x), f(a.y), f(a.z), f(a.w));
}
template <class F>
__device__ __forceinline__ float4 zip4(float4 a, float4 b, F f) {
    return make_float4(f(a.x, b.x), f(a.y, b.y), f(a.z, b.z), f(a.w, b.w));
}

// v plus lane-permuted v, both halves of the double through DPP.
template <int kCtrl>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kCtrl, 0xF, 0xF, false);
    return v + __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// Sum over the wave, wave-uniform (the moves of row16_max: within pairs, within
// quads, halves of 8 mirrored, the row of 16 mirrored, then the four rows).
__device__ __forceinline__ double wave_sum(double v) {
    v = dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Sum and maximum over the workgroup's T threads, the same in every thread.
// `slot` is LDS not used by the previous reduction (one barrier per reduction,
// none for a workgroup of one wave).
template <int T>
__device__ __forceinline__ double block_sum(double v, double *slot) {
    v = wave_sum(v);
    if constexpr (T == 64) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += slot[w];
    return v;
}

template <int T>
__device__ __forceinline__ float block_max(float v, float *slot) {
    v = wave_max(v);
    if constexpr (T == 64) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = fmaxf(v, slot[w]);
    return v;
}

// The row (NV float4 per thread, zeros past n4) out: fp32, bf16, or its codes
// and scale as s3d8_quant_act makes them.
template <int T, int NV>
__device__ __forceinline__ void row_out(const float4 (&v)[NV], int64_t row, int K, int out_type, void *rows, int8_t *xq,
                                        float *xs, float *slot) {
    const int n4 = K >> 2;
    if (out_type != S3D8_ROWS_CODES) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * T;
            if (i < n4) store4(rows, row * K + 4 * i, v[j], out_type == S3D8_ROWS_BF16);
        }
        return;
    }
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        a = fmaxf(a, fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)), fmaxf(fabsf(v[j].z), fabsf(v[j].w))));
    a = block_max<T>(a, slot);
    const float s = a / 127.0f;
    if (threadIdx.x == 0) xs[row] = s;
    // The code is rne(fl(x / s)).  t = x fl(1 / s) differs from x / s by less than
    // 127 2^-23, fl(x / s) by less than 127 2^-24: where t is further than 2^-15
    // from a border k + 1/2, rne(t) is the code.  A thread with a value nearer
    // than that (or with 1 / s infinite) divides.
    const float rs = 1.0f / s;
    bool divide = false;
    uint32_t q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const float x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        q[j] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float t = x[e] * rs, k = rintf(t);
            divide |= !(fabsf(t - k) <= 0.5f - 0x1p-15f);
            q[j] |= (uint32_t)((int)k & 0xFF) << (8 * e);
        }
    }
    if (divide) {
        auto code = [&](float x) {
            return a == 0.0f ? 0u : (uint32_t)(uint8_t)(int8_t)fminf(127.0f, fmaxf(-127.0f, rintf(x / s)));
        };
#pragma unroll
        for (int j = 0; j < NV; ++j)
            q[j] = code(v[j].x) | code(v[j].y) << 8 | code(v[j].z) << 16 | code(v[j].w) << 24;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + j * T;
        if (i < n4) reinterpret_cast<uint32_t *>(xq + row * K)[i] = q[j];
    }
}

// N(v; w, b) of a row.  The statistics are sums of exact products in 64 bits,
// rounded to fp32 once: an fp32 sum would depend on its order, and its last
// bit moves codes across their rounding borders.
template <int T, int NV>
__device__ __forceinline__ void normalise(float4 (&v)[NV], int K, bool layer, float eps, const float *__restrict__ w,
                                          const float *__restrict__ b, double *slot) {
    const int n4 = K >> 2;
    double mu = 0.0;
    if (layer) {
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j) s += ((double)v[j].x + (double)v[j].y) + ((double)v[j].z + (double)v[j].w);
        mu = block_sum<T>(s, slot) / (double)K;
        slot += T / 64;
    }
    double q = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if ((int)threadIdx.x + j * T < n4) {  // (past the row v is 0, not mu)
            const double x = v[j].x - mu, y = v[j].y - mu, z = v[j].z - mu, t = v[j].w - mu;
            q += (x * x + y * y) + (z * z + t * t);
        }
    }
    const float r = (float)(1.0 / sqrt(block_sum<T>(q, slot) / (double)K + (double)eps));
    const float m = (float)mu;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + j * T;
        if (i >= n4) continue;
        float4 u = v[j];
        if (layer) u = map4(u, [&](float x) { return x - m; });
        u = zip4(map4(u, [&](float x) { return x * r; }), reinterpret_cast<const float4 *>(w)[i],
                 [](float x, float y) { return x * y; });
        if (b) u = zip4(u, reinterpret_cast<const float4 *>(b)[i], [](float x, float y) { return x + y; });
        v[j] = u;
    }
}

// One workgroup per row.
template <int T, int NV>
__global__ __launch_bounds__(T) void block_norm_kernel(const s3d8_block_norm_args p) {
    __shared__ double sums[4][T / 64];
    __shared__ float maxima[T / 64];
    const int64_t row = blockIdx.x;
    const int K = (int)p.K, n4 = K >> 2;
    const bool layer = p.kind == S3D8_NORM_LAYER;
    float4 h[NV];
    load_row<T, NV>(h, p.h, row * K, n4, p.h_type == S3D8_ROWS_BF16);
    if (p.branch) {
        float4 b[NV];
        load_row<T, NV>(b, p.branch, row * K, n4, p.branch_type == S3D8_ROWS_BF16);
        if (p.post_weight) normalise<T, NV>(b, K, layer, p.eps, p.post_weight, p.post_bias, sums[0]);
        const float rs = p.residual_scale;
        auto factor = [&](float g) { return p.gate_tanh ? (float)tanh((double)g) : g; };
        const float g1 = p.gate && !p.gate_channels ? factor(*p.gate) : 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * T;
            if (i >= n4) continue;
            float4 t = b[j];
            if (p.gate && p.gate_channels)
                t = zip4(map4(reinterpret_cast<const float4 *>(p.gate)[i], factor), t,
                         [](float g, float x) { return g * x; });
            else
                t = map4(t, [&](float x) { return g1 * x; });
            h[j] = zip4(h[j], t, [&](float x, float y) { return rs * x + y; });
            if (p.h_type == S3D8_ROWS_BF16) {
                // the norm reads the residual as it is stored
                const uint2 u = bf16x4(h[j]);
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.h_out) + row * K + 4 * i) = u;
                h[j] = bf16x4_values(u);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(p.h_out) + row * K + 4 * i) = h[j];
            }
        }
    }
    normalise<T, NV>(h, K, layer, p.eps, p.weight, p.bias, sums[2]);
    row_out<T, NV>(h, row, K, p.out_type, p.rows, p.xq, p.xs, maxima);
}

// SiLU(g) * u = g u / (1 + exp(-g)) in 64 bits, rounded to fp32 once, to a
// relative 2^-50 before that (so that it is the correctly rounded product but
// for one value in some 2^25).  exp: -g = n ln 2 + r with ln 2 in two parts, a
// degree-11 polynomial on |r| <= ln 2 / 2 (Chebyshev interpolation, relative
// error 2^-55.7), 2^n by ldexp.  |g| is cut at 700, where the result is already
// g u or, below 2^-149, a zero of its sign; the denominator stays finite.
// The quotient: two Newton steps on the hardware reciprocal.
// About 31 instructions against some 80 of the library's exp and division.
__device__ __forceinline__ float gated(float g, float u) {
    const double x = (double)-__builtin_amdgcn_fmed3f(g, -700.0f, 700.0f);
    const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
    const double r = __builtin_fma(n, -0x1.a39ef35793c76p-33, __builtin_fma(n, -0x1.62e42fee00000p-1, x));
    double e = 0x1.af631d203b4edp-26;
    e = __builtin_fma(e, r, 0x1.28b405992d897p-22);
    e = __builtin_fma(e, r, 0x1.71ddf5748bd71p-19);
    e = __builtin_fma(e, r, 0x1.a01991ac6b2ddp-16);
    e = __builtin_fma(e, r, 0x1.a01a01b1437f6p-13);
    e = __builtin_fma(e, r, 0x1.6c16c187fbea9p-10);
    e = __builtin_fma(e, r, 0x1.111111110f225p-7);
    e = __builtin_fma(e, r, 0x1.555555554f0cep-5);
    e = __builtin_fma(e, r, 0x1.555555555555ap-3);
    e = __builtin_fma(e, r, 0x1.0000000000011p-1);
    e = __builtin_fma(e, r, 1.0);
    e = __builtin_fma(e, r, 1.0);
    const double d = 1.0 + __builtin_amdgcn_ldexp(e, (int)n), a = (double)g * (double)u;
    double q = __builtin_amdgcn_rcp(d);
    q = __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
    q = __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
    return (float)(a * q);
}

template <int T, int NV>
__global__ __launch_bounds__(T) void glu_act_kernel(const void *__restrict__ gate, int64_t ldg,
                                                    const void *__restrict__ up, int64_t ldu, int K, int in_bf,
                                                    int out_type, void *__restrict__ rows, int8_t *__restrict__ xq,
                                                    float *__restrict__ xs) {
    __shared__ float maxima[T / 64];
    const int64_t row = blockIdx.x;
    const int n4 = K >> 2;
    float4 v[NV], u[NV];
    load_row<T, NV>(v, gate, row * ldg, n4, in_bf);
    load_row<T, NV>(u, up, row * ldu, n4, in_bf);
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if ((int)threadIdx.x + j * T < n4) v[j] = zip4(v[j], u[j], gated);
    row_out<T, NV>(v, row, K, out_type, rows, xq, xs, maxima);
}

// --------------------------------------------------------------- host

struct BlockNorm {
    template <int T, int NV>
    static constexpr auto kernel() { return &block_norm_kernel<T, NV>; }
};
struct GluAct {
    template <int T, int NV>
    static constexpr auto kernel() { return &glu_act_kernel<T, NV>; }
};

template <class Op, int T>
auto row_kernel_of(int64_t nv) {
    switch (nv) {
        case 1: return Op::template kernel<T, 1>();
        case 2: return Op::template kernel<T, 2>();
        case 3: return Op::template kernel<T, 3>();
        case 4: return Op::template kernel<T, 4>();
        case 5: return Op::template kernel<T, 5>();
        case 6: return Op::template kernel<T, 6>();
        case 7: return Op::template kernel<T, 7>();
        default: return Op::template kernel<T, 8>();
    }
}

// The workgroup of a row: where there are rows for every CU, the fewest threads
// that hold it in 8 float4 each (few waves to join, many rows on a CU); else as
// many as it has float4 (short chains).
template <class Op>
auto row_kernel(int64_t M, int64_t K, int cus, int &threads) {
    const int64_t n4 = K / 4;
    auto nv = [&](int t) { return (n4 + t - 1) / t; };
    const int64_t most = M >= 2 * cus ? 8 : 1;
    if (nv(64) <= most) return threads = 64, row_kernel_of<Op, 64>(nv(64));
    if (nv(256) <= most) return threads = 256, row_kernel_of<Op, 256>(nv(256));
    if (nv(512) <= most) return threads = 512, row_kernel_of<Op, 512>(nv(512));
    threads = 1024;
    return nv(1024) <= 8 ? row_kernel_of<Op, 1024>(nv(1024)) : Op::template kernel<1024, 16>();
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_rows(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0) return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (K % 16 != 0) return s3d8::fail(S3D8_ERR_SHAPE, "K must be a multiple of 16");
    if (K > kMaxWidth) return s3d8::fail(S3D8_ERR_SHAPE, "K over 65536 is not supported");
    if (M > kMaxRows) return s3d8::fail(S3D8_ERR_SHAPE, "more than 524288 rows are not supported");
    return S3D8_OK;
}

bool row_type(int32_t t) { return t == S3D8_ROWS_F32 || t == S3D8_ROWS_BF16; }

int check_out(int32_t out_type, const void *rows, const int8_t *xq, const float *xs) {
    if (!row_type(out_type) && out_type != S3D8_ROWS_CODES)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown output type");
    const bool codes = out_type == S3D8_ROWS_CODES;
    if (codes ? rows || !xq || !xs : !rows || xq || xs)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "codes need xq and xs and no rows, other outputs rows alone");
    if (!aligned(rows, 16) || !aligned(xq, 16))
        return s3d8::fail(S3D8_ERR_ALIGN, "output rows and xq must be 16-byte aligned");
    if (!aligned(xs, 4)) return s3d8::fail(S3D8_ERR_ALIGN, "xs must be 4-byte aligned");
    return S3D8_OK;
}

}  // namespace

extern "C" {

int32_t s3d8_block_norm(const s3d8_block_norm_args *args, void *stream) {
    if (!args || !args->h || !args->weight) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    const s3d8_block_norm_args &a = *args;
    if ((a.branch != nullptr) != (a.h_out != nullptr))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "h_out goes with branch");
    if (!a.branch && (a.post_weight || a.gate))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "a post norm or gate needs a branch");
    if (a.kind != S3D8_NORM_RMS && a.kind != S3D8_NORM_LAYER)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown norm kind");
    if (a.kind == S3D8_NORM_RMS && (a.bias || a.post_bias))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "an RMS norm has no bias");
    if (a.post_bias && !a.post_weight) return s3d8::fail(S3D8_ERR_INVALID_ARG, "post_bias needs post_weight");
    if (!row_type(a.h_type) || (a.branch && !row_type(a.branch_type)))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    if (!(a.eps > 0.0f)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "eps must be positive");
    int rc = check_rows(a.M, a.K);
    if (rc) return rc;
    rc = check_out(a.out_type, a.rows, a.xq, a.xs);
    if (rc) return rc;
    if (!aligned(a.h, 16) || !aligned(a.branch, 16) || !aligned(a.h_out, 16) || !aligned(a.weight, 16) ||
        !aligned(a.bias, 16) || !aligned(a.post_weight, 16) || !aligned(a.post_bias, 16) ||
        !aligned(a.gate, a.gate_channels ? 16 : 4))
        return s3d8::fail(S3D8_ERR_ALIGN, "rows and [K] vectors must be 16-byte aligned");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    int threads = 0;
    const auto fn = row_kernel<BlockNorm>(a.M, a.K, cus, threads);
    hipLaunchKernelGGL(fn, dim3((unsigned)a.M), dim3(threads), 0, (hipStream_t)stream, a);
    return s3d8::launch_status();
}

int32_t s3d8_glu_act(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int64_t M, int64_t K,
                     int32_t in_type, int32_t out_type, void *rows, int8_t *xq, float *xs, void *stream) {
    if (!gate || !up) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    if (!row_type(in_type)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    int rc = check_rows(M, K);
    if (rc) return rc;
    rc = check_out(out_type, rows, xq, xs);
    if (rc) return rc;
    const int64_t lim = int64_t(1) << 40;
    if (ld_gate < K || ld_up < K || ld_gate > lim || ld_up > lim)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "row strides must be at least K (and below 2^40)");
    const uintptr_t four = in_type == S3D8_ROWS_F32 ? 16 : 8;
    if (ld_gate % 4 || ld_up % 4 || !aligned(gate, four) || !aligned(up, four))
        return s3d8::fail(S3D8_ERR_ALIGN, "gate and up rows must be aligned to 4 elements");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    int threads = 0;
    const auto fn = row_kernel<GluAct>(M, K, cus, threads);
    hipLaunchKernelGGL(fn, dim3((unsigned)M), dim3(threads), 0, (hipStream_t)stream, gate, ld_gate, up, ld_up,
                       (int)K, (int)(in_type == S3D8_ROWS_BF16), out_type, rows, xq, xs);
    return s3d8::launch_status();
}

}  // extern "C"
