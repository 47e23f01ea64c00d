// norm_residual.cu -- the norms after and before a block, fused with the
// block's gate and the residual scale (moe_norm_residual), and its gradients
// (moe_norm_residual_backward).
//
//   n  = gamma_post * y * rp,           rp = 1 / sqrt(mean(y^2) + eps)
//   h' = a h + g * n                    a: residual scale, g: gate
//   u  = gamma_pre * h' * rq,           rq = 1 / sqrt(mean(h'^2) + eps)
//
// u comes from the unrounded fp32 h' (h' is rounded once, when it is stored):
// the next block's input then carries one rounding, not two.
//
// Backward, with q = du * gamma_pre, hn = h' rq, yn = y rp:
//   D  = dh' + rq (q - hn * mean(q hn))
//   dh = a D,   dg = D * gamma_post * yn
//   p  = D * g * gamma_post,   dy = rp (p - yn * mean(p yn))
//   dgamma_post = sum_t D g yn,   dgamma_pre = sum_t du hn,   dg summed over t for a gate per channel
// mean(p yn) needs D, which needs mean(q hn); expanding D makes both come out
// of one reduction over three sums:
//   sum(p yn) = sum(w (dh' + rq q)) - rq mean(q hn) sum(w hn),   w = g gamma_post yn
#include "moe.h"
#include "kernels.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>

namespace moe {
moe_status_t api_fail(moe_status_t st, const char* msg);
void api_clear_error();
moe_status_t api_sm_count(int* n);
}  // namespace moe

namespace {

constexpr int kNrMaxH = 16384;
constexpr int kNrBwdBlocks = 148;   // row walkers of the backward pass, one partial sum each

struct NrArgs {
    const uint16_t *h, *y, *gamma_post, *gate, *gamma_pre;
    float a, eps;
    int T, H, gate_mode;
    uint16_t *h_out, *u;
    float* rstd;                       // [2, T]: rp, rq
    // backward
    const float* rstd_in;
    const uint16_t *dh_out, *du;
    uint16_t *dh, *dy;
    void* dgate;                       // fp32 [H] (channel) or bf16 [T, H] (token)
    float *dgamma_post, *dgamma_pre;
    float* part;                       // [blocks][3][H]
    int blocks;
};

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ const uint4* vec(const uint16_t* p, size_t row, int H) {
    return reinterpret_cast<const uint4*>(p + row * H);
}

// Sum of N values over the block in a fixed order, on every thread.  `sh`
// holds N * 32 floats; consecutive calls must use different halves.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
        if (lane == 0) sh[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = lane < nw ? sh[i * 32 + lane] : 0.0f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        v[i] = s;
    }
}

__device__ __forceinline__ float inv_norm(float ss, int H, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps)));
}

// One block per row; a thread keeps NV 8-value vectors of the row in registers.
template <int NV>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const NrArgs p) {
    __shared__ float sh[2][32];
    const int nvec = p.H / 8;
    const size_t t = blockIdx.x;
    uint4 yr[NV], hr[NV];
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        yr[i] = c < nvec ? vec(p.y, t, p.H)[c] : make_uint4(0, 0, 0, 0);
        hr[i] = c < nvec ? vec(p.h, t, p.H)[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[8];
        unpack8(yr[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = fmaf(f[j], f[j], ss[0]);
    }
    block_sum(ss, sh[0]);
    const float rp = inv_norm(ss[0], p.H, p.eps);
    float h2[NV][8];
    float s2[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h2[i][j] = 0.0f;
            continue;
        }
        float y[8], h[8], g[8], w[8];
        unpack8(yr[i], y);
        unpack8(hr[i], h);
        unpack8(__ldg(vec(p.gamma_post, 0, p.H) + c), w);
        if (p.gate_mode == MOE_GATE_NONE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = 1.0f;
        } else {
            unpack8(__ldg(vec(p.gate, p.gate_mode == MOE_GATE_TOKEN ? t : 0, p.H) + c), g);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h2[i][j] = fmaf(g[j], w[j] * (y[j] * rp), p.a * h[j]);
            s2[0] = fmaf(h2[i][j], h2[i][j], s2[0]);
        }
        reinterpret_cast<uint4*>(p.h_out + t * p.H)[c] = pack8(h2[i]);
    }
    if (p.u == nullptr) {
        if (threadIdx.x == 0 && p.rstd) p.rstd[t] = rp;
        return;
    }
    block_sum(s2, sh[1]);
    const float rq = inv_norm(s2[0], p.H, p.eps);
    if (threadIdx.x == 0 && p.rstd) {
        p.rstd[t] = rp;
        p.rstd[p.T + t] = rq;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        float w[8], o[8];
        unpack8(__ldg(vec(p.gamma_pre, 0, p.H) + c), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = w[j] * (h2[i][j] * rq);
        reinterpret_cast<uint4*>(p.u + t * p.H)[c] = pack8(o);
    }
}

// Persistent blocks walk rows blockIdx.x, blockIdx.x + blocks, ...; a thread
// owns the same columns in every row, so the column sums stay in its
// registers and leave as one partial per block.
template <int NV>
__global__ void __launch_bounds__(1024) norm_residual_bwd_kernel(const NrArgs p) {
    __shared__ float sh[2][3 * 32];
    const int nvec = p.H / 8;
    const float inv_h = 1.0f / (float)p.H;
    float sgp[NV][8], sgq[NV][8], sg[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sgp[i][j] = sgq[i][j] = sg[i][j] = 0.0f;
    int half = 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    for (size_t t = blockIdx.x; t < (size_t)p.T; t += gridDim.x) {
        const float rp = p.rstd_in[t], rq = p.du ? p.rstd_in[p.T + t] : 0.0f;
        uint4 yr[NV], hr[NV], dr[NV], ur[NV], gr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const bool ok = c < nvec;
            yr[i] = ok ? vec(p.y, t, p.H)[c] : zero;
            hr[i] = ok ? vec(p.h, t, p.H)[c] : zero;
            dr[i] = ok ? vec(p.dh_out, t, p.H)[c] : zero;
            ur[i] = ok && p.du ? vec(p.du, t, p.H)[c] : zero;
            gr[i] = one;
            if (ok && p.gate_mode != MOE_GATE_NONE)
                gr[i] = vec(p.gate, p.gate_mode == MOE_GATE_TOKEN ? t : 0, p.H)[c];
        }
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float y[8], h[8], d[8], u[8], g[8], wp[8], wq[8];
            unpack8(yr[i], y);
            unpack8(hr[i], h);
            unpack8(dr[i], d);
            unpack8(ur[i], u);
            unpack8(gr[i], g);
            unpack8(__ldg(vec(p.gamma_post, 0, p.H) + c), wp);
            unpack8(p.gamma_pre ? __ldg(vec(p.gamma_pre, 0, p.H) + c) : zero, wq);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = g[j] * (wp[j] * (y[j] * rp));
                const float hn = fmaf(p.a, h[j], w) * rq;
                const float q = u[j] * wq[j];
                s[0] = fmaf(q, hn, s[0]);
                s[1] = fmaf(w, fmaf(rq, q, d[j]), s[1]);
                s[2] = fmaf(w, hn, s[2]);
            }
        }
        block_sum(s, sh[half]);
        half ^= 1;
        const float c1 = s[0] * inv_h;
        const float c2 = (s[1] - rq * c1 * s[2]) * inv_h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float y[8], h[8], d[8], u[8], g[8], wp[8], wq[8], odh[8], ody[8], odg[8];
            unpack8(yr[i], y);
            unpack8(hr[i], h);
            unpack8(dr[i], d);
            unpack8(ur[i], u);
            unpack8(gr[i], g);
            unpack8(__ldg(vec(p.gamma_post, 0, p.H) + c), wp);
            unpack8(p.gamma_pre ? __ldg(vec(p.gamma_pre, 0, p.H) + c) : zero, wq);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float yn = y[j] * rp;
                const float hn = fmaf(p.a, h[j], g[j] * (wp[j] * yn)) * rq;
                const float D = fmaf(rq, fmaf(u[j], wq[j], -hn * c1), d[j]);
                const float Dg = D * g[j];
                odh[j] = p.a * D;
                ody[j] = rp * fmaf(Dg, wp[j], -yn * c2);
                odg[j] = D * (wp[j] * yn);
                sgp[i][j] = fmaf(Dg, yn, sgp[i][j]);
                sgq[i][j] = fmaf(u[j], hn, sgq[i][j]);
                sg[i][j] += odg[j];
            }
            reinterpret_cast<uint4*>(p.dh + t * p.H)[c] = pack8(odh);
            reinterpret_cast<uint4*>(p.dy + t * p.H)[c] = pack8(ody);
            if (p.gate_mode == MOE_GATE_TOKEN)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dgate) + t * p.H)[c] = pack8(odg);
        }
    }
    float* base = p.part + (size_t)blockIdx.x * 3 * p.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            *reinterpret_cast<float4*>(base + 8 * c + j) =
                make_float4(sgp[i][j], sgp[i][j + 1], sgp[i][j + 2], sgp[i][j + 3]);
            *reinterpret_cast<float4*>(base + p.H + 8 * c + j) =
                make_float4(sgq[i][j], sgq[i][j + 1], sgq[i][j + 2], sgq[i][j + 3]);
            *reinterpret_cast<float4*>(base + 2 * p.H + 8 * c + j) =
                make_float4(sg[i][j], sg[i][j + 1], sg[i][j + 2], sg[i][j + 3]);
        }
    }
}

// Column sums of the per-block partials in block order, in binary64.
__global__ void __launch_bounds__(256) norm_residual_cols_kernel(const NrArgs p) {
    __shared__ double sh[8][33];
    const int which = blockIdx.y;
    float* out = which == 0 ? p.dgamma_post : which == 1 ? p.dgamma_pre : static_cast<float*>(p.dgate);
    if (which == 2 && p.gate_mode != MOE_GATE_CHANNEL) return;
    if (out == nullptr) return;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    double s = 0.0;
    if (col < p.H)
        for (int b = w; b < p.blocks; b += 8) s += (double)p.part[((size_t)b * 3 + which) * p.H + col];
    sh[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && col < p.H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sh[i][threadIdx.x];
        out[col] = (float)s;
    }
}

// Threads of a block: one 8-value vector each up to 1024 threads, then as few
// vectors each as cover the row.
struct NrShape {
    int nv, threads;
};
NrShape nr_shape(int H) {
    const int nvec = H / 8;
    const int nv = (nvec + 1023) / 1024;
    return {nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}

moe_status_t nfail(moe_status_t st, const char* fmt, const char* a, long long b = 0) {
    char msg[192];
    snprintf(msg, sizeof(msg), fmt, a, b);
    return moe::api_fail(st, msg);
}

#define NR_TRY(x)                          \
    do {                                   \
        moe_status_t st_ = (x);            \
        if (st_ != MOE_OK) return st_;     \
    } while (0)

moe_status_t need(const void* p, const char* name, size_t align) {
    if (!p) return nfail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return nfail(MOE_ERR_INVALID_ARG, "%s must be %lld-byte aligned", name, (long long)align);
    return MOE_OK;
}

moe_status_t check_shape(const moe_config_t* c) {
    if (!c) return moe::api_fail(MOE_ERR_INVALID_ARG, "config is NULL");
    if (c->T < 0) return nfail(MOE_ERR_INVALID_ARG, "%s=%lld must be >= 0", "T", c->T);
    if (c->H <= 0 || c->H % 8 || c->H > kNrMaxH)
        return nfail(MOE_ERR_UNSUPPORTED, "%s=%lld must be a multiple of 8 in [8, 16384]", "H", c->H);
    return MOE_OK;
}

moe_status_t check_common(const moe_config_t* c, const void* h, const void* y, const void* gamma_post,
                          const void* gate, int32_t gate_mode, float a) {
    if (c->T > 0) {  // with no rows the row buffers may be empty (NULL)
        NR_TRY(need(h, "h", 16));
        NR_TRY(need(y, "y", 16));
    }
    NR_TRY(need(gamma_post, "gamma_post", 16));
    if (gate_mode != MOE_GATE_NONE && gate_mode != MOE_GATE_CHANNEL && gate_mode != MOE_GATE_TOKEN)
        return nfail(MOE_ERR_INVALID_ARG, "unknown %s %lld", "gate_mode", gate_mode);
    if (gate_mode == MOE_GATE_NONE) {
        if (gate) return moe::api_fail(MOE_ERR_INVALID_ARG, "gate given with MOE_GATE_NONE");
    } else if (c->T > 0 || gate_mode == MOE_GATE_CHANNEL) {
        NR_TRY(need(gate, "gate", 16));
    }
    if (!std::isfinite(a)) return moe::api_fail(MOE_ERR_INVALID_ARG, "res_scale must be finite");
    return MOE_OK;
}

// An output over an input is fine where both start at the same address and the
// documentation allows it; any other overlap is refused.
bool overlap(const void* p, size_t pb, const void* q, size_t qb) {
    const char *a = static_cast<const char*>(p), *b = static_cast<const char*>(q);
    return a && b && a < b + qb && b < a + pb;
}

moe_status_t launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return MOE_OK;
    return nfail(MOE_ERR_CUDA, what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

moe_status_t moe_norm_residual(const moe_config_t* cfg, const void* h, const void* y,
                               const void* gamma_post, const void* gate, int32_t gate_mode,
                               float res_scale, float eps, const void* gamma_pre, void* h_out,
                               void* u, float* rstd, moe_stream_t stream) {
    moe::api_clear_error();
    NR_TRY(check_shape(cfg));
    NR_TRY(check_common(cfg, h, y, gamma_post, gate, gate_mode, res_scale));
    if (!(eps >= 0.0f) || !(eps < 1e30f))
        return moe::api_fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (cfg->T == 0) return MOE_OK;
    NR_TRY(need(h_out, "h_out", 16));
    if ((gamma_pre == nullptr) != (u == nullptr))
        return moe::api_fail(MOE_ERR_INVALID_ARG, "gamma_pre and u must be given together");
    if (u) {
        NR_TRY(need(gamma_pre, "gamma_pre", 16));
        NR_TRY(need(u, "u", 16));
    }
    const size_t n = (size_t)cfg->T * cfg->H * 2;
    if (overlap(u, n, h, n) || overlap(u, n, h_out, n) || (u != y && overlap(u, n, y, n)))
        return moe::api_fail(MOE_ERR_INVALID_ARG, "u overlaps h, h_out or part of y");
    if ((h_out != h && overlap(h_out, n, h, n)) || overlap(h_out, n, y, n))
        return moe::api_fail(MOE_ERR_INVALID_ARG, "h_out overlaps y or part of h");
    if (gate_mode == MOE_GATE_TOKEN && (overlap(h_out, n, gate, n) || overlap(u, n, gate, n)))
        return moe::api_fail(MOE_ERR_INVALID_ARG, "h_out or u overlaps the gate");
    if (rstd) NR_TRY(need(rstd, "rstd", 4));
    NrArgs p = {};
    p.h = static_cast<const uint16_t*>(h);
    p.y = static_cast<const uint16_t*>(y);
    p.gamma_post = static_cast<const uint16_t*>(gamma_post);
    p.gate = static_cast<const uint16_t*>(gate);
    p.gamma_pre = static_cast<const uint16_t*>(gamma_pre);
    p.a = res_scale;
    p.eps = eps;
    p.T = cfg->T;
    p.H = cfg->H;
    p.gate_mode = gate_mode;
    p.h_out = static_cast<uint16_t*>(h_out);
    p.u = static_cast<uint16_t*>(u);
    p.rstd = rstd;
    const NrShape sh = nr_shape(p.H);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (sh.nv == 1)
        norm_residual_kernel<1><<<p.T, sh.threads, 0, s>>>(p);
    else
        norm_residual_kernel<2><<<p.T, sh.threads, 0, s>>>(p);
    return launched("norm_residual launch: %s");
}

size_t moe_norm_residual_workspace_size(const moe_config_t* cfg) {
    moe::api_clear_error();
    if (check_shape(cfg) != MOE_OK) return 0;
    return (size_t)kNrBwdBlocks * 3 * cfg->H * 4;
}

moe_status_t moe_norm_residual_backward(const moe_config_t* cfg, const void* h, const void* y,
                                        const void* gamma_post, const void* gate,
                                        int32_t gate_mode, float res_scale, const void* gamma_pre,
                                        const float* rstd, const void* dh_out, const void* du,
                                        void* dh, void* dy, void* dgate, float* dgamma_post,
                                        float* dgamma_pre, void* ws, size_t ws_bytes,
                                        moe_stream_t stream) {
    moe::api_clear_error();
    NR_TRY(check_shape(cfg));
    NR_TRY(check_common(cfg, h, y, gamma_post, gate, gate_mode, res_scale));
    const bool rows = cfg->T > 0;
    if (rows) {
        NR_TRY(need(rstd, "rstd", 4));
        NR_TRY(need(dh_out, "dh_out", 16));
        NR_TRY(need(dh, "dh", 16));
        NR_TRY(need(dy, "dy", 16));
    }
    NR_TRY(need(dgamma_post, "dgamma_post", 16));
    if ((gamma_pre == nullptr) != (dgamma_pre == nullptr) || (rows && (gamma_pre == nullptr) != (du == nullptr)))
        return moe::api_fail(MOE_ERR_INVALID_ARG, "gamma_pre, du and dgamma_pre must be given together");
    if (gamma_pre) {
        NR_TRY(need(gamma_pre, "gamma_pre", 16));
        NR_TRY(need(dgamma_pre, "dgamma_pre", 16));
        if (rows) NR_TRY(need(du, "du", 16));
    }
    if (gate_mode == MOE_GATE_NONE && dgate)
        return moe::api_fail(MOE_ERR_INVALID_ARG, "dgate given with MOE_GATE_NONE");
    if (gate_mode == MOE_GATE_CHANNEL || (gate_mode == MOE_GATE_TOKEN && rows)) NR_TRY(need(dgate, "dgate", 16));
    const size_t n = (size_t)cfg->T * cfg->H * 2;
    const void* token_gate = gate_mode == MOE_GATE_TOKEN ? gate : nullptr;
    const void* token_dgate = gate_mode == MOE_GATE_TOKEN ? dgate : nullptr;
    const struct { const void* p; const char* name; const void* may; } outs[] = {
        {dh, "dh", dh_out}, {dy, "dy", du}, {token_dgate, "dgate", token_gate}};
    for (const auto& o : outs) {
        for (const void* in : {h, y, dh_out, du, token_gate})
            if (in != o.may ? overlap(o.p, n, in, n) : o.p != in && overlap(o.p, n, in, n))
                return nfail(MOE_ERR_INVALID_ARG, "%s overlaps an input", o.name);
        for (const auto& q : outs)
            if (&q != &o && overlap(o.p, n, q.p, n))
                return nfail(MOE_ERR_INVALID_ARG, "%s overlaps another output", o.name);
    }
    NR_TRY(need(ws, "workspace", 256));
    const size_t bytes = (size_t)kNrBwdBlocks * 3 * cfg->H * 4;
    if (ws_bytes < bytes)
        return nfail(MOE_ERR_WORKSPACE, "workspace too small, %s %lld bytes", "needs", (long long)bytes);
    NrArgs p = {};
    p.h = static_cast<const uint16_t*>(h);
    p.y = static_cast<const uint16_t*>(y);
    p.gamma_post = static_cast<const uint16_t*>(gamma_post);
    p.gate = static_cast<const uint16_t*>(gate);
    p.gamma_pre = static_cast<const uint16_t*>(gamma_pre);
    p.a = res_scale;
    p.T = cfg->T;
    p.H = cfg->H;
    p.gate_mode = gate_mode;
    p.rstd_in = rstd;
    p.dh_out = static_cast<const uint16_t*>(dh_out);
    p.du = static_cast<const uint16_t*>(du);
    p.dh = static_cast<uint16_t*>(dh);
    p.dy = static_cast<uint16_t*>(dy);
    p.dgate = dgate;
    p.dgamma_post = dgamma_post;
    p.dgamma_pre = dgamma_pre;
    p.part = static_cast<float*>(ws);
    p.blocks = cfg->T < kNrBwdBlocks ? cfg->T : kNrBwdBlocks;
    const NrShape sh = nr_shape(p.H);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.T > 0) {
        if (sh.nv == 1)
            norm_residual_bwd_kernel<1><<<p.blocks, sh.threads, 0, s>>>(p);
        else
            norm_residual_bwd_kernel<2><<<p.blocks, sh.threads, 0, s>>>(p);
        NR_TRY(launched("norm_residual backward launch: %s"));
    }
    // with no rows the sums are zero
    norm_residual_cols_kernel<<<dim3((p.H + 31) / 32, 3), 256, 0, s>>>(p);
    return launched("norm_residual column-sum launch: %s");
}

}  // extern "C"
