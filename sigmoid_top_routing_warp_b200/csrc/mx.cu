// mx.cu -- MXFP4 weights (moe_quantize_mx, moe_dequantize_mx): blocks of 32
// values along a row share one power-of-two scale (e8m0, one byte) and hold
// a 4-bit e2m1 code each (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign).
//
//   scale = 2^(floor(log2 amax) - 2)      (2: the exponent of e2m1's largest value 6 = 1.5 * 2^2)
//   code  = e2m1(x / scale), round to nearest even, saturating at 6
//
// The scale needs no logarithm: floor(log2) of a bf16 amax is its exponent
// field, so the e8m0 byte is max(field, 2) - 2 (bytes below 0 clamp to 0), 127
// for an all-zero block and 255 (NaN) when the block holds an infinity or a
// NaN.  x / scale is a product with a power of two, exact in binary32, so the
// only rounding is the conversion's.
//
// Both directions only move bytes: 2 B read and 0.53 B written per value, or
// the reverse.  163840 x 1536, there and back: 196 us for 1.27 GB, 6.5 TB/s, as
// fast as a copy (202 to 205 in a loop of calls; a small matrix is two launches,
// 10 us).  The matrix is dense and a row is a multiple of 32, so it is walked as
// one flat array: a lane owns 8 values (a 16-byte access on the bf16 side, 4
// bytes of codes), four lanes a block, and every lane keeps
// kMxVecs accesses in flight.
#include "moe.h"
#include "kernels.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdio>

namespace moe {
moe_status_t api_fail(moe_status_t st, const char* msg);
void api_clear_error();
}  // namespace moe

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxVecs = 4;                              // 8-value vectors in flight per thread
constexpr long long kMxPerBlock = (long long)kMxThreads * kMxVecs;

// two binary32 values -> two e2m1 codes (lo in bits 0-3)
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// two e2m1 codes (bits 0-7 of c) -> two binary16 values
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t c) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(c));
    return r;
}

__global__ void __launch_bounds__(kMxThreads) quantize_mx_kernel(const uint4* __restrict__ x, long long nvec,
                                                                 uint32_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scale) {
    const long long v0 = (long long)blockIdx.x * kMxPerBlock + threadIdx.x;
    uint4 raw[kMxVecs];
#pragma unroll
    for (int i = 0; i < kMxVecs; ++i) {
        const long long v = v0 + i * kMxThreads;
        raw[i] = v < nvec ? __ldcs(x + v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kMxVecs; ++i) {
        const long long v = v0 + i * kMxThreads;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        // magnitudes compare as integers
        uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                               __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
        const uint32_t amax = max(m2 & 0xffffu, m2 >> 16);
        const uint32_t field = amax >> 7;
        const uint32_t s = amax == 0 ? 127u : field == 255u ? 255u : max(field, 2u) - 2u;
        // 1 / scale = 2^(127 - s): s is at most 252 here, so the factor is normal
        const float inv = s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
        uint32_t code = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
            code |= e2m1x2(__fmul_rn(lo, inv), __fmul_rn(hi, inv)) << (8 * j);
        }
        if (v < nvec) {
            q[v] = s == 255u ? 0u : code;
            if ((threadIdx.x & 3) == 0) scale[v >> 2] = (uint8_t)s;
        }
    }
}

__global__ void __launch_bounds__(kMxThreads) dequantize_mx_kernel(const uint32_t* __restrict__ q,
                                                                   const uint8_t* __restrict__ scale,
                                                                   long long nvec, uint4* __restrict__ x) {
    const long long v0 = (long long)blockIdx.x * kMxPerBlock + threadIdx.x;
    uint32_t code[kMxVecs], s[kMxVecs];
#pragma unroll
    for (int i = 0; i < kMxVecs; ++i) {
        const long long v = v0 + i * kMxThreads;
        code[i] = v < nvec ? __ldcs(q + v) : 0u;
        s[i] = v < nvec ? (uint32_t)__ldg(scale + (v >> 2)) : 127u;
    }
#pragma unroll
    for (int i = 0; i < kMxVecs; ++i) {
        const long long v = v0 + i * kMxThreads;
        // 2^(s - 127): 2^-127 is subnormal, 255 stands for NaN
        const float f = __uint_as_float(s[i] == 0u ? 0x00400000u : s[i] == 255u ? 0x7fc00000u : s[i] << 23);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h = e2m1x2_to_f16x2(code[i] >> (8 * j));
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
            const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(p.x, f), __fmul_rn(p.y, f));
            o[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (v < nvec) __stcs(x + v, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

moe_status_t mx_check(const void* x, const void* q, const void* scale, int32_t rows, int32_t cols) {
    char msg[160];
    if (rows < 0 || cols < 0 || cols % 32) {
        snprintf(msg, sizeof(msg), "rows=%d must be >= 0, cols=%d a multiple of 32", rows, cols);
        return moe::api_fail(MOE_ERR_INVALID_ARG, msg);
    }
    if (rows == 0 || cols == 0) return MOE_OK;
    const struct { const void* p; const char* name; size_t align; } arg[] = {
        {x, "x", 16}, {q, "q", 16}, {scale, "scale", 1}};
    for (const auto& a : arg) {
        if (!a.p) {
            snprintf(msg, sizeof(msg), "%s is NULL", a.name);
            return moe::api_fail(MOE_ERR_INVALID_ARG, msg);
        }
        if (reinterpret_cast<uintptr_t>(a.p) % a.align) {
            snprintf(msg, sizeof(msg), "%s must be %zu-byte aligned", a.name, a.align);
            return moe::api_fail(MOE_ERR_INVALID_ARG, msg);
        }
    }
    const size_t n = (size_t)rows * cols;
    const moe::Span span[] = {{x, 2 * n, "x"}, {q, n / 2, "q"}, {scale, n / 32, "scale"}};
    for (int i = 0; i < 3; ++i)
        if (moe::overlap(span[i], span[(i + 1) % 3])) {
            snprintf(msg, sizeof(msg), "%s overlaps %s", span[i].name, span[(i + 1) % 3].name);
            return moe::api_fail(MOE_ERR_INVALID_ARG, msg);
        }
    return MOE_OK;
}

moe_status_t mx_launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return MOE_OK;
    char msg[160];
    snprintf(msg, sizeof(msg), "%s launch: %s", what, cudaGetErrorString(e));
    return moe::api_fail(MOE_ERR_CUDA, msg);
}

// The grid stays below 2^31 blocks of 8192 values for up to 2^44 values, more
// than a GPU holds.
unsigned mx_grid(long long nvec) { return (unsigned)((nvec + kMxPerBlock - 1) / kMxPerBlock); }

}  // namespace

extern "C" {

moe_status_t moe_quantize_mx(const void* x, int32_t rows, int32_t cols, uint8_t* q, uint8_t* scale,
                             moe_stream_t stream) {
    moe::api_clear_error();
    const moe_status_t st = mx_check(x, q, scale, rows, cols);
    if (st != MOE_OK) return st;
    const long long nvec = (long long)rows * cols / 8;
    if (nvec == 0) return MOE_OK;
    quantize_mx_kernel<<<mx_grid(nvec), kMxThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(x), nvec, reinterpret_cast<uint32_t*>(q), scale);
    return mx_launched("MXFP4 quantisation");
}

moe_status_t moe_dequantize_mx(const uint8_t* q, const uint8_t* scale, int32_t rows, int32_t cols,
                               void* x, moe_stream_t stream) {
    moe::api_clear_error();
    const moe_status_t st = mx_check(x, q, scale, rows, cols);
    if (st != MOE_OK) return st;
    const long long nvec = (long long)rows * cols / 8;
    if (nvec == 0) return MOE_OK;
    dequantize_mx_kernel<<<mx_grid(nvec), kMxThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<const uint32_t*>(q), scale, nvec, static_cast<uint4*>(x));
    return mx_launched("MXFP4 read-back");
}

}  // extern "C"
