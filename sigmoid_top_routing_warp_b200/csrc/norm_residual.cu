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
// Without the norm after the update D = dh', and h has no part in anything.
//
// Both are bound by HBM and by the latency of a row's sums (load, sum over the
// block, store), which rows copied ahead into shared memory hide in part:
//   forward   8192 x 5120, gate per token: 82 us for 420 MB, 5.1 TB/s (a copy
//             runs at 6.53); 4 x 5120: 8 us, a launch
//   backward  8192 x 5120, gate per channel: 98 us for 503 MB, 5.1 TB/s, 74 us
//             for 336 MB without the norm after the update (97 when it read h
//             all the same); 777 x 4096, gate per token: 22 us for 51 MB, two
//             launches, the second one's start hidden behind the first (27 us
//             without that)
// Tried and not kept: the next row's loads issued across the sum (126-140 us
// for the backward, registers), four rows in flight, 256-byte L2 fetches and
// streaming stores (no change), column sums of 148 partials by blocks of 1024
// threads (+2 us), pairs of rows with one sum in 640 threads (121 us).
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
constexpr int kNrWideThreads = 512;
constexpr int kNrWideSmem = 220 << 10;   // for its rows
constexpr int kNrBwdThreads = 384; // of a block of the backward pass at most: one or two 8-value vectors each
constexpr int kNrBwdShort = 2560;  // columns up to which they have one
constexpr int kNrBwdBlocks = 148;   // row walkers of the backward pass, one partial sum each; several times as
                                    // many for short rows

// Threads of a block of the backward pass, and most blocks of it.  A block works
// on one row at a time and waits for its sum, so an SM gets as many as 640
// threads hold, up to eight: 8192 rows of 2560 / 1024 / 256 columns take 58 / 33 /
// 20 us (with one block an SM, before h was left out where it has no part, 83 /
// 65 / 58, with several 62 / 34 / 22).  Two vectors a thread from 2560 columns on:
// 2560 with two 80 us and with one 82 in one block an SM, 1024 67 and 63.
int bwd_threads(int H) {
    const int vecs = H / 8;
    return ((H <= kNrBwdShort ? vecs : (vecs + 1) / 2) + 31) / 32 * 32;
}
int bwd_blocks(int H) {
    if (H > kNrBwdShort) return kNrBwdBlocks;
    const int n = 640 / bwd_threads(H);
    return kNrBwdBlocks * (n < 8 ? n : 8);
}

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
    float* part;                       // [blocks][2][H]
    int blocks;
};

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

// 16 bytes from global to this thread's own place in shared memory.  Only the
// thread that issued a copy reads it back, behind copies_left: no barrier.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// The column sums are launched as a programmatic dependent: their blocks come
// up while the rows are still worked on, and wait here for the end of that
// kernel, whose writes they then see.
__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of the closed groups are still under way
template <int N>
__device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

// Two binary32 operations in one instruction (the same bits as two).
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split(F2 a, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 widen(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t narrow(F2 a) {
    float x, y;
    split(a, x, y);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float total(F2 a) {
    float x, y;
    split(a, x, y);
    return x + y;
}

constexpr int kNrStages = 3;       // rows in a block's shared memory: one worked on, the others on their way

// Blocks walk rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread keeps NV
// 8-value vectors of the row, ST rows of them in shared memory.
template <int NV, int ST, int THREADS, bool TOKEN>
__global__ void __launch_bounds__(THREADS, 1280 / THREADS) norm_residual_kernel(const NrArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sh[2][2][32];
    constexpr int NT = TOKEN ? 3 : 2;                 // tensors of a row: y, h, gate
    const int nvec = p.H / 8, nthr = blockDim.x;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    auto place = [&](int st, int k, int i) { return mine + ((st * NT + k) * NV + i) * nthr * 16; };
    auto fetch = [&](size_t t, int st) {
        if (t < (size_t)p.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = threadIdx.x + i * nthr;
                const bool ok = c < nvec;
                const int cc = ok ? c : 0;
                copy16(place(st, 0, i), vec(p.y, t, p.H) + cc, ok);
                copy16(place(st, 1, i), vec(p.h, t, p.H) + cc, ok);
                if (TOKEN) copy16(place(st, 2, i), vec(p.gate, t, p.H) + cc, ok);
            }
        }
        copies_close();
    };
    size_t t = blockIdx.x;
    const size_t step = gridDim.x;
#pragma unroll
    for (int d = 0; d < ST - 1; ++d) fetch(t + d * step, d);
    const F2 a2 = f2(p.a, p.a);
    int st = 0, half = 0;
    for (; t < (size_t)p.T; t += step, half ^= 1) {
        copies_left<ST - 2>();
        uint4 yr[NV], hr[NV], gr[NV];
        F2 ss = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            yr[i] = lds128(place(st, 0, i));
            hr[i] = lds128(place(st, 1, i));
            if (TOKEN) gr[i] = lds128(place(st, 2, i));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const F2 y = widen(word(yr[i], j));
                ss = fma2(y, y, ss);
            }
        }
        fetch(t + (ST - 1) * step, st == 0 ? ST - 1 : st - 1);   // the row before this one has left its place
        st = st == ST - 1 ? 0 : st + 1;
        float s1[1] = {total(ss)};
        block_sum(s1, sh[half][0]);
        const float rp = inv_norm(s1[0], p.H, p.eps);
        const F2 rp2 = f2(rp, rp);
        F2 h2[NV][4], s2 = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * nthr;
            const bool ok = c < nvec;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint4 w = ok ? __ldg(vec(p.gamma_post, 0, p.H) + c) : zero;
            if (!TOKEN) gr[i] = ok && p.gate ? __ldg(vec(p.gate, 0, p.H) + c)
                                             : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const F2 n = widen(word(w, j)) * (widen(word(yr[i], j)) * rp2);
                h2[i][j] = fma2(widen(word(gr[i], j)), n, a2 * widen(word(hr[i], j)));
                s2 = fma2(h2[i][j], h2[i][j], s2);
                o[j] = narrow(h2[i][j]);
            }
            if (ok) reinterpret_cast<uint4*>(p.h_out + t * p.H)[c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (p.u == nullptr) {
            if (threadIdx.x == 0 && p.rstd) p.rstd[t] = rp;
            continue;
        }
        float s3[1] = {total(s2)};
        block_sum(s3, sh[half][1]);
        const float rq = inv_norm(s3[0], p.H, p.eps);
        if (threadIdx.x == 0 && p.rstd) {
            p.rstd[t] = rp;
            p.rstd[p.T + t] = rq;
        }
        const F2 rq2 = f2(rq, rq);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * nthr;
            if (c >= nvec) continue;
            const uint4 w = __ldg(vec(p.gamma_pre, 0, p.H) + c);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = narrow(widen(word(w, j)) * (h2[i][j] * rq2));
            reinterpret_cast<uint4*>(p.u + t * p.H)[c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Tensors of a row that the backward pass reads: y, dh_out, with the norm after
// the update h and du, with a gate per token the gate.
constexpr int row_tensors(bool token, bool pre) { return 2 + (pre ? 2 : 0) + (token ? 1 : 0); }

// Persistent blocks, NV 8-value vectors of the row per thread; a thread owns
// the same columns in every row, so the column sums stay in its registers and
// leave as one partial per block.  A gate per channel and no gate are constant
// down a column, so sum(D yn) alone gives both dgamma_post (times g) and dgate
// (times gamma_post); with a gate per token it is sum(D g yn).  Without the
// norm after the update (PRE) D is dh' alone: h is not read, and an infinity or
// a NaN in it reaches no gradient.
template <int NV, bool TOKEN, bool PRE>
__global__ void __launch_bounds__(kNrBwdThreads) norm_residual_bwd_kernel(const NrArgs p) {
    let_dependents_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sh[2][3 * 32];
    constexpr int NT = row_tensors(TOKEN, PRE), kGate = NT - 1;   // of a row: y, dh_out, with PRE h and du, gate
    const int nthr = blockDim.x, nvec = p.H / 8;
    const float inv_h = 1.0f / (float)p.H;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    auto place = [&](int st, int k, int i) { return mine + ((st * NT + k) * NV + i) * nthr * 16; };
    auto fetch = [&](size_t t, int st) {
        if (t < (size_t)p.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = threadIdx.x + i * nthr;
                const bool ok = c < nvec;
                const int cc = ok ? c : 0;
                copy16(place(st, 0, i), vec(p.y, t, p.H) + cc, ok);
                copy16(place(st, 1, i), vec(p.dh_out, t, p.H) + cc, ok);
                if (PRE) {
                    copy16(place(st, 2, i), vec(p.h, t, p.H) + cc, ok);
                    copy16(place(st, 3, i), vec(p.du, t, p.H) + cc, ok);
                }
                if (TOKEN) copy16(place(st, kGate, i), vec(p.gate, t, p.H) + cc, ok);
            }
        }
        copies_close();
    };
    size_t t = blockIdx.x;
    const size_t step = gridDim.x;
    fetch(t, 0);
    fetch(t + step, 1);
    // the columns' weights; a gate that is the same in every row is part of wp
    F2 wp[NV][4], wq[NV][4], sp[NV][4], sq[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nthr;
        const bool ok = c < nvec;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        const uint4 w1 = ok ? __ldg(vec(p.gamma_post, 0, p.H) + c) : zero;
        const uint4 w2 = PRE && ok ? __ldg(vec(p.gamma_pre, 0, p.H) + c) : zero;
        const uint4 gc = ok && p.gate_mode == MOE_GATE_CHANNEL ? __ldg(vec(p.gate, 0, p.H) + c) : one;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            wp[i][j] = TOKEN ? widen(word(w1, j)) : widen(word(gc, j)) * widen(word(w1, j));
            wq[i][j] = widen(word(w2, j));
            sp[i][j] = sq[i][j] = f2(0.0f, 0.0f);
        }
    }
    const F2 a2 = f2(p.a, p.a);
    int st = 0, half = 0;
    float rp_next = __ldg(p.rstd_in + t), rq_next = PRE ? __ldg(p.rstd_in + p.T + t) : 0.0f;
    for (; t < (size_t)p.T; t += step) {
        const float rp = rp_next, rq = rq_next;
        const F2 rp2 = f2(rp, rp), rq2 = f2(rq, rq);
        copies_left<1>();
        if (t + step < (size_t)p.T) {
            rp_next = __ldg(p.rstd_in + t + step);
            rq_next = PRE ? __ldg(p.rstd_in + p.T + t + step) : 0.0f;
        }
        F2 yn[NV][4], hn[NV][4], dq[NV][4];           // dq: dh' + rq q
        uint4 gr[NV];
        F2 x0 = f2(0.0f, 0.0f), x1 = x0, x2 = x0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4 yr = lds128(place(st, 0, i)), dr = lds128(place(st, 1, i));
            uint4 hr, ur;
            if (PRE) {
                hr = lds128(place(st, 2, i));
                ur = lds128(place(st, 3, i));
            }
            if (TOKEN) gr[i] = lds128(place(st, kGate, i));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                yn[i][j] = widen(word(yr, j)) * rp2;
                F2 w = wp[i][j] * yn[i][j];
                if (TOKEN) w = widen(word(gr[i], j)) * w;
                dq[i][j] = widen(word(dr, j));
                if (PRE) {
                    hn[i][j] = fma2(a2, widen(word(hr, j)), w) * rq2;
                    const F2 u = widen(word(ur, j));
                    const F2 q = u * wq[i][j];
                    dq[i][j] = fma2(rq2, q, dq[i][j]);
                    x0 = fma2(q, hn[i][j], x0);
                    x2 = fma2(w, hn[i][j], x2);
                    sq[i][j] = fma2(u, hn[i][j], sq[i][j]);
                }
                x1 = fma2(w, dq[i][j], x1);
            }
        }
        fetch(t + 2 * step, st == 0 ? kNrStages - 1 : st - 1);
        st = st == kNrStages - 1 ? 0 : st + 1;
        float s[PRE ? 3 : 1] = {total(x1)};
        if constexpr (PRE) {
            s[1] = total(x0);
            s[2] = total(x2);
        }
        block_sum(s, sh[half]);
        half ^= 1;
        float c1 = 0.0f, c2 = s[0] * inv_h;
        if constexpr (PRE) {
            c1 = s[1] * inv_h;
            c2 = (s[0] - rq * c1 * s[2]) * inv_h;
        }
        const F2 k1 = f2(-rq * c1, -rq * c1), k2 = f2(-c2, -c2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * nthr;
            uint32_t odh[4], ody[4], odg[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const F2 D = PRE ? fma2(hn[i][j], k1, dq[i][j]) : dq[i][j];
                const F2 Dg = TOKEN ? D * widen(word(gr[i], j)) : D;
                odh[j] = narrow(a2 * D);
                ody[j] = narrow(rp2 * fma2(yn[i][j], k2, Dg * wp[i][j]));
                if (TOKEN) odg[j] = narrow(D * (wp[i][j] * yn[i][j]));
                sp[i][j] = fma2(Dg, yn[i][j], sp[i][j]);
            }
            if (c >= nvec) continue;
            reinterpret_cast<uint4*>(p.dh + t * p.H)[c] = make_uint4(odh[0], odh[1], odh[2], odh[3]);
            reinterpret_cast<uint4*>(p.dy + t * p.H)[c] = make_uint4(ody[0], ody[1], ody[2], ody[3]);
            if (TOKEN)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dgate) + t * p.H)[c] =
                    make_uint4(odg[0], odg[1], odg[2], odg[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nthr;
        if (c >= nvec) continue;
        float* base = p.part + (size_t)blockIdx.x * 2 * p.H + 8 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x, y;
            split(sp[i][j], x, y);
            *reinterpret_cast<float2*>(base + 2 * j) = make_float2(x, y);
            if (PRE) {
                split(sq[i][j], x, y);
                *reinterpret_cast<float2*>(base + p.H + 2 * j) = make_float2(x, y);
            }
        }
    }
}

// Rows of more than 6144 columns, up to 512 threads: only the column sums stay
// in registers.  A row stays in shared memory until its second pass, which
// computes the first one's values again (128 registers a thread hold no more),
// and the columns' weights come from L1.  ST rows are there or on their way.
// 4096 x 8192: 109 us (403 MB, 62 us of copies), 131 in 1024 threads with half the
// vectors, 230 with both passes from L2; 2048 x 16384: 129. Without the norm after
// the update 84 and 75.
template <int NV, int ST, bool TOKEN, bool PRE>
__global__ void __launch_bounds__(kNrWideThreads) norm_residual_bwd_wide_kernel(const NrArgs p) {
    let_dependents_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sh[2][3 * 32];
    constexpr int NT = row_tensors(TOKEN, PRE), kGate = NT - 1;   // of a row: y, dh_out, with PRE h and du, gate
    const int nthr = blockDim.x, nvec = p.H / 8;
    const float inv_h = 1.0f / (float)p.H;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    auto place = [&](int st, int k, int i) { return mine + ((st * NT + k) * NV + i) * nthr * 16; };
    auto fetch = [&](size_t t, int st) {
        if (t < (size_t)p.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = threadIdx.x + i * nthr;
                const bool ok = c < nvec;
                const int cc = ok ? c : 0;
                copy16(place(st, 0, i), vec(p.y, t, p.H) + cc, ok);
                copy16(place(st, 1, i), vec(p.dh_out, t, p.H) + cc, ok);
                if (PRE) {
                    copy16(place(st, 2, i), vec(p.h, t, p.H) + cc, ok);
                    copy16(place(st, 3, i), vec(p.du, t, p.H) + cc, ok);
                }
                if (TOKEN) copy16(place(st, kGate, i), vec(p.gate, t, p.H) + cc, ok);
            }
        }
        copies_close();
    };
    size_t t = blockIdx.x;
    const size_t step = gridDim.x;
#pragma unroll
    for (int k = 0; k < ST; ++k) fetch(t + k * step, k);
    F2 sp[NV][4], sq[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sp[i][j] = sq[i][j] = f2(0.0f, 0.0f);
    const F2 a2 = f2(p.a, p.a);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int st = 0, half = 0;
    for (; t < (size_t)p.T; t += step) {
        const float rp = __ldg(p.rstd_in + t), rq = PRE ? __ldg(p.rstd_in + p.T + t) : 0.0f;
        const F2 rp2 = f2(rp, rp), rq2 = f2(rq, rq);
        // a vector of the row: both passes take the same values from it
        auto values = [&](int i, auto use) {
            const int c = threadIdx.x + i * nthr;
            const bool ok = c < nvec;
            const uint4 w1 = ok ? __ldg(vec(p.gamma_post, 0, p.H) + c) : zero;
            const uint4 w2 = PRE && ok ? __ldg(vec(p.gamma_pre, 0, p.H) + c) : zero;
            uint4 gr;
            if (TOKEN)
                gr = lds128(place(st, kGate, i));
            else
                gr = ok && p.gate_mode == MOE_GATE_CHANNEL ? __ldg(vec(p.gate, 0, p.H) + c)
                                                           : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
            const uint4 yr = lds128(place(st, 0, i)), dr = lds128(place(st, 1, i));
            uint4 hr, ur;
            if (PRE) {
                hr = lds128(place(st, 2, i));
                ur = lds128(place(st, 3, i));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const F2 g = widen(word(gr, j)), wg = widen(word(w1, j));
                const F2 yn = widen(word(yr, j)) * rp2, w = g * (wg * yn);
                F2 hn = f2(0.0f, 0.0f), u = hn, q = hn, dq = widen(word(dr, j));
                if (PRE) {
                    hn = fma2(a2, widen(word(hr, j)), w) * rq2;
                    u = widen(word(ur, j));
                    q = u * widen(word(w2, j));
                    dq = fma2(rq2, q, dq);
                }
                use(j, g, wg, yn, w, hn, u, q, dq);
            }
        };
        copies_left<ST - 1>();
        F2 x0 = f2(0.0f, 0.0f), x1 = x0, x2 = x0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            values(i, [&](int j, F2, F2, F2, F2 w, F2 hn, F2 u, F2 q, F2 dq) {
                x1 = fma2(w, dq, x1);
                if (PRE) {
                    x0 = fma2(q, hn, x0);
                    x2 = fma2(w, hn, x2);
                    sq[i][j] = fma2(u, hn, sq[i][j]);
                }
            });
        float s[PRE ? 3 : 1] = {total(x1)};
        if constexpr (PRE) {
            s[1] = total(x0);
            s[2] = total(x2);
        }
        block_sum(s, sh[half]);
        half ^= 1;
        float c1 = 0.0f, c2 = s[0] * inv_h;
        if constexpr (PRE) {
            c1 = s[1] * inv_h;
            c2 = (s[0] - rq * c1 * s[2]) * inv_h;
        }
        const F2 k1 = f2(-rq * c1, -rq * c1), k2 = f2(-c2, -c2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * nthr;
            uint32_t odh[4], ody[4], odg[4];
            values(i, [&](int j, F2 g, F2 wg, F2 yn, F2, F2 hn, F2, F2, F2 dq) {
                const F2 D = PRE ? fma2(hn, k1, dq) : dq;
                const F2 Dg = D * g;
                odh[j] = narrow(a2 * D);
                ody[j] = narrow(rp2 * fma2(yn, k2, Dg * wg));
                if (TOKEN) odg[j] = narrow(D * (wg * yn));
                // a gate per channel is a factor of the whole column
                sp[i][j] = fma2(TOKEN ? Dg : D, yn, sp[i][j]);
            });
            if (c >= nvec) continue;
            reinterpret_cast<uint4*>(p.dh + t * p.H)[c] = make_uint4(odh[0], odh[1], odh[2], odh[3]);
            reinterpret_cast<uint4*>(p.dy + t * p.H)[c] = make_uint4(ody[0], ody[1], ody[2], ody[3]);
            if (TOKEN)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dgate) + t * p.H)[c] =
                    make_uint4(odg[0], odg[1], odg[2], odg[3]);
        }
        fetch(t + ST * step, st);
        if (ST > 1) st = st == ST - 1 ? 0 : st + 1;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nthr;
        if (c >= nvec) continue;
        float* base = p.part + (size_t)blockIdx.x * 2 * p.H + 8 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x, y;
            split(sp[i][j], x, y);
            *reinterpret_cast<float2*>(base + 2 * j) = make_float2(x, y);
            if (PRE) {
                split(sq[i][j], x, y);
                *reinterpret_cast<float2*>(base + p.H + 2 * j) = make_float2(x, y);
            }
        }
    }
}

// Column sums of the per-block partials in block order, in binary64:
// blockIdx.y 0 gives dgamma_post and a channel gate's dgate, 1 dgamma_pre.
template <int NW>   // warps, each with a share of the partials
__global__ void __launch_bounds__(NW * 32) norm_residual_cols_kernel(const NrArgs p) {
    __shared__ double sh[NW][33];
    const int which = blockIdx.y;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    after_primary();
    double s = 0.0;
    if (col < p.H) {
#pragma unroll 8
        for (int b = w; b < p.blocks; b += NW) s += (double)p.part[((size_t)b * 2 + which) * p.H + col];
    }
    sh[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w != 0 || col >= p.H) return;
#pragma unroll
    for (int i = 1; i < NW; ++i) s += sh[i][threadIdx.x];
    if (which == 1) {
        p.dgamma_pre[col] = (float)s;
    } else if (p.gate_mode == MOE_GATE_CHANNEL && p.blocks > 0) {   // (of no rows an infinite factor makes nothing)
        p.dgamma_post[col] = (float)(s * (double)__uint_as_float((uint32_t)p.gate[col] << 16));
        static_cast<float*>(p.dgate)[col] = (float)(s * (double)__uint_as_float((uint32_t)p.gamma_post[col] << 16));
    } else {
        p.dgamma_post[col] = (float)s;
        if (p.gate_mode == MOE_GATE_CHANNEL) static_cast<float*>(p.dgate)[col] = (float)s;
    }
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

// An output, and the input that it may be: an overlap with anything else is
// refused, and with that input one that does not start where it does.
struct Out {
    moe::Span s;
    const void* may;
};
template <int NI, int NO>
moe_status_t apart(const moe::Span (&in)[NI], const Out (&outs)[NO]) {
    for (const Out& o : outs) {
        for (const moe::Span& i : in)
            if (moe::overlap(o.s, i) && !(i.p == o.may && i.p == o.s.p))
                return nfail(MOE_ERR_INVALID_ARG, "%s overlaps an input", o.s.name);
        for (const Out& q : outs)
            if (&q != &o && moe::overlap(o.s, q.s)) return nfail(MOE_ERR_INVALID_ARG, "%s overlaps another output", o.s.name);
    }
    return MOE_OK;
}

moe_status_t launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return MOE_OK;
    return nfail(MOE_ERR_CUDA, what, cudaGetErrorString(e));
}

// A kernel's limit of dynamic shared memory is the process's: always the most
// that its variant takes, or a call of another size in another thread could
// lower it between this and the launch.
template <class Kernel>
cudaError_t smem_limit(Kernel* kernel, int most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

template <int NV, int ST, int THREADS, bool TOKEN>
moe_status_t launch_forward(const NrArgs& p, int threads, cudaStream_t s) {
    auto* kernel = norm_residual_kernel<NV, ST, THREADS, TOKEN>;
    constexpr int per_thread = ST * (TOKEN ? 3 : 2) * NV * 16;
    const int smem = per_thread * threads;
    int sms = 0, fit = 1;
    NR_TRY(moe::api_sm_count(&sms));
    cudaError_t e = smem_limit(kernel, per_thread * THREADS);
    if (e == cudaSuccess && p.T > sms) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, smem);
    if (e != cudaSuccess) return nfail(MOE_ERR_CUDA, "norm_residual: %s", cudaGetErrorString(e));
    const int most = sms * (fit > 0 ? fit : 1);
    kernel<<<p.T < most ? p.T : most, threads, smem, s>>>(p);
    return launched("norm_residual launch: %s");
}

// One 8-value vector a thread, two above 8192 columns, and as many blocks of
// an SM as registers and shared memory hold: with one block of 640 threads the
// SM idles while it waits for a row's sums (8192 rows of 5120: 131 us against
// 82 with two).
template <bool TOKEN>
moe_status_t run_forward(const NrArgs& p, cudaStream_t s) {
    const int nvec = p.H / 8, nv = nvec <= 1024 ? 1 : 2;
    const int threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    if (nv == 2) return launch_forward<2, 2, 1024, TOKEN>(p, threads, s);
    if (threads <= 320) return launch_forward<1, kNrStages, 320, TOKEN>(p, threads, s);
    if (threads <= 640) return launch_forward<1, kNrStages, 640, TOKEN>(p, threads, s);
    return launch_forward<1, kNrStages, 1024, TOKEN>(p, threads, s);
}

template <int NV, bool TOKEN, bool PRE>
moe_status_t launch_backward(const NrArgs& p, cudaStream_t s) {
    const int threads = bwd_threads(p.H);
    constexpr int per_thread = kNrStages * row_tensors(TOKEN, PRE) * NV * 16;
    const int smem = per_thread * threads;
    const cudaError_t e = smem_limit(norm_residual_bwd_kernel<NV, TOKEN, PRE>, per_thread * kNrBwdThreads);
    if (e != cudaSuccess) return nfail(MOE_ERR_CUDA, "norm_residual backward: %s", cudaGetErrorString(e));
    norm_residual_bwd_kernel<NV, TOKEN, PRE><<<p.blocks, threads, smem, s>>>(p);
    return MOE_OK;
}

// Two rows in shared memory where they fit, up to 11 or 13 thousand columns
// (without the norm after the update they always do: three tensors of 16384
// columns are 96 KB).
template <bool TOKEN, bool PRE>
moe_status_t launch_backward_wide(const NrArgs& p, cudaStream_t s) {
    const int nv = p.H <= 16 * kNrWideThreads ? 2 : 4;
    const int threads = ((p.H / 8 + nv - 1) / nv + 31) / 32 * 32;
    const int row = row_tensors(TOKEN, PRE) * nv * threads * 16;
    const int st = !PRE || 2 * row <= kNrWideSmem ? 2 : 1;
    auto* kernel = nv == 2 ? norm_residual_bwd_wide_kernel<2, 2, TOKEN, PRE> : norm_residual_bwd_wide_kernel<4, 2, TOKEN, PRE>;
    if constexpr (PRE)
        if (st == 1) kernel = norm_residual_bwd_wide_kernel<4, 1, TOKEN, PRE>;
    const cudaError_t e = smem_limit(kernel, kNrWideSmem);
    if (e != cudaSuccess) return nfail(MOE_ERR_CUDA, "norm_residual backward: %s", cudaGetErrorString(e));
    kernel<<<p.blocks, threads, st * row, s>>>(p);
    return MOE_OK;
}

template <bool TOKEN, bool PRE>
moe_status_t run_backward(const NrArgs& p, cudaStream_t s) {
    if (p.H <= kNrBwdShort) return launch_backward<1, TOKEN, PRE>(p, s);
    if (p.H <= 16 * kNrBwdThreads) return launch_backward<2, TOKEN, PRE>(p, s);
    return launch_backward_wide<TOKEN, PRE>(p, s);
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
    if (rstd) NR_TRY(need(rstd, "rstd", 4));
    const size_t row = (size_t)cfg->H * 2, n = cfg->T * row;
    const moe::Span in[] = {{h, n, "h"},
                            {y, n, "y"},
                            {gamma_post, row, "gamma_post"},
                            {gate, gate_mode == MOE_GATE_TOKEN ? n : row, "gate"},
                            {gamma_pre, row, "gamma_pre"}};
    const Out outs[] = {{{h_out, n, "h_out"}, h}, {{u, n, "u"}, y}, {{rstd, (size_t)cfg->T * (u ? 8 : 4), "rstd"}, nullptr}};
    NR_TRY(apart(in, outs));
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return gate_mode == MOE_GATE_TOKEN ? run_forward<true>(p, s) : run_forward<false>(p, s);
}

size_t moe_norm_residual_workspace_size(const moe_config_t* cfg) {
    moe::api_clear_error();
    if (check_shape(cfg) != MOE_OK) return 0;
    return (size_t)bwd_blocks(cfg->H) * 2 * cfg->H * 4;
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
    NR_TRY(need(ws, "workspace", 256));
    const size_t bytes = (size_t)bwd_blocks(cfg->H) * 2 * cfg->H * 4;
    if (ws_bytes < bytes)
        return nfail(MOE_ERR_WORKSPACE, "workspace too small, %s %lld bytes", "needs", (long long)bytes);
    const bool token = gate_mode == MOE_GATE_TOKEN;
    const size_t row = (size_t)cfg->H * 2, n = cfg->T * row;
    const moe::Span in[] = {{h, n, "h"},
                            {y, n, "y"},
                            {gamma_post, row, "gamma_post"},
                            {gate, token ? n : row, "gate"},
                            {gamma_pre, row, "gamma_pre"},
                            {rstd, (size_t)cfg->T * (gamma_pre ? 8 : 4), "rstd"},
                            {dh_out, n, "dh_out"},
                            {gamma_pre ? du : nullptr, n, "du"}};
    const Out outs[] = {{{dh, n, "dh"}, dh_out},
                        {{dy, n, "dy"}, du},
                        {{dgate, token ? n : 2 * row, "dgate"}, token ? gate : nullptr},
                        {{dgamma_post, 2 * row, "dgamma_post"}, nullptr},
                        {{dgamma_pre, 2 * row, "dgamma_pre"}, nullptr},
                        {{ws, bytes, "workspace"}, nullptr}};
    NR_TRY(apart(in, outs));
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
    // eight rows of a block and more, where that leaves a block for every SM
    p.blocks = cfg->T / 8 < bwd_blocks(cfg->H) ? cfg->T / 8 : bwd_blocks(cfg->H);
    if (p.blocks < kNrBwdBlocks) p.blocks = cfg->T < kNrBwdBlocks ? cfg->T : kNrBwdBlocks;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.T > 0) {
        if (du)
            NR_TRY((token ? run_backward<true, true>(p, s) : run_backward<false, true>(p, s)));
        else
            NR_TRY((token ? run_backward<true, false>(p, s) : run_backward<false, false>(p, s)));
        NR_TRY(launched("norm_residual backward launch: %s"));
    }
    // with no rows the sums are zero
    cudaLaunchConfig_t cols = {};
    cols.gridDim = dim3((p.H + 31) / 32, dgamma_pre ? 2 : 1);
    const bool many = p.blocks > kNrBwdBlocks;
    cols.blockDim = dim3(many ? 1024 : 256);
    cols.stream = s;
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cols.attrs = &early;
    cols.numAttrs = p.T > 0 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cols, many ? norm_residual_cols_kernel<32> : norm_residual_cols_kernel<8>, p);
    if (e != cudaSuccess) return nfail(MOE_ERR_CUDA, "norm_residual column-sum launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

}  // extern "C"
