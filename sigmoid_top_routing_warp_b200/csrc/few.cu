// few.cu -- the whole MoE FFN layer for a few tokens in one launch
// (moe_forward_few): router, choice, the experts' SwiGLU and the combine.
//
// Steps a1-a9 of the layer (sources in include/moe.h).  One cooperative
// launch, one block per SM, three phases with two grid barriers between them:
//   R   router logits: a warp per (expert, K slice)
//   1   every block repeats the choice (T * E keys) and builds the plan of
//       touched experts in shared memory, then gate/up rows and SwiGLU
//   2   down rows; a row sums over its token's experts in a fixed order
#include "moe.h"
#include "kernels.cuh"
#include "tiles.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdio>

namespace moe {
moe_status_t api_check_config(const moe_config_t* c);
moe_status_t api_fail(moe_status_t st, const char* msg);
void api_clear_error();
moe_status_t api_sm_count(int* n);
}  // namespace moe

namespace {

constexpr int kT = MOE_FEW_MAX_T;
constexpr int kMaxE = 1024, kMaxK = 32;
constexpr int kMaxPairs = kT * (kMaxK + 1);      // (expert, token) pairs, the shared expert's among them
constexpr int kMaxActive = kT * kMaxK + 1;       // touched experts and the shared one
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBarWord = moe::kSchedFirstWord;   // grid barriers (2) and the exit count, in the status block

struct FewArgs {
    const uint16_t *x, *w_router;
    const float* bias;
    const uint8_t *w13, *w2, *w13s, *w2s;
    const void *s13, *s2, *s13s, *s2s;
    uint16_t* out;
    int32_t* idx;
    float* w;
    int* status;
    double* part;      // [n_split][T][E] logits of the K slices
    float* act;        // [pairs][max(I, Is)] weighted SwiGLU outputs
    int T, H, E, k, I, Is, n_group, topk_group, group_topn, norm, n_split, stall, ld_act;
    float rsf;
};

// The touched experts, the same in every block.
struct Plan {
    int n_active;
    int expert[kMaxActive];         // -1: the shared expert
    uint32_t mask[kMaxActive];      // its tokens
    int base[kMaxActive];           // its first pair
    float w[kMaxPairs];             // routing weight of a pair
    int sel[kT * kMaxK];            // the choice [T, k]
    float selw[kT * kMaxK];
    uint32_t emask[kMaxE];          // tokens of each expert
    int apos[kMaxE];                // an expert's place in the list
    int abort;
};

// (key, index) order of the choice: larger key first, then lower index.
__device__ __forceinline__ bool better(double a, int ia, double b, int ib) {
    return a > b || (a == b && ia < ib);
}
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const double ov = __shfl_xor_sync(0xffffffffu, v, off);
        const int oi = __shfl_xor_sync(0xffffffffu, i, off);
        if (better(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    }
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Grid barrier `b`, used once per launch: every block arrives, then waits for
// the count.  Bounded; false when it gave up.
__device__ bool grid_barrier(const FewArgs& a, int b, volatile int* abort_flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        int* bar = a.status + kBarWord + b;
        __threadfence();
        if (!(a.stall && b == 0 && blockIdx.x == 0)) atomicAdd(bar, 1);
        const long long t0 = clock64();
        while (*reinterpret_cast<volatile int*>(bar) < (int)gridDim.x) {
            if (clock64() - t0 > moe::kWaitLimit) {
                atomicOr(a.status, moe::DEV_STATUS_TIMEOUT);
                *abort_flag = 1;
                break;
            }
        }
        __threadfence();
    }
    __syncthreads();
    return *abort_flag == 0;
}

// e8m0 scale byte -> binary32 (0 is 2^-127, 255 NaN)
__device__ __forceinline__ float e8m0(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
}

// Weights k .. k + 7 of row `row` of a matrix with K columns (whose first row
// is `w`, scales `s`) in binary32.
template <int DT>
__device__ __forceinline__ void load8(const uint8_t* w, const void* s, size_t row, int K, int k, float* f) {
    if (DT == MOE_DTYPE_BF16) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + (row * K + k) * 2)), f);
    } else if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(w + row * K + k));
        const float sc = __ldg(static_cast<const float*>(s) + (row / 128) * (K / 128) + k / 128);
        const uint32_t c[2] = {v.x, v.y};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            __nv_fp8_e4m3 q;
            q.__x = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
            f[i] = (float)q * sc;
        }
    } else {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(w + (row * K + k) / 2));
        const float sc = e8m0(__ldg(static_cast<const uint8_t*>(s) + (row * K + k) / 32));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = v >> (4 * i) & 15u, e = c >> 1 & 3u, m = c & 1u;
            const float mag = e ? (float)((2u + m) << (e - 1)) * 0.5f : 0.5f * (float)m;
            f[i] = (c & 8u ? -mag : mag) * sc;
        }
    }
}

// Phase R: logits of expert e over one K slice, one warp each.  Eight exact
// products are summed in binary32, those sums in binary64: the logit's error
// stays near 2^-25 of a partial sum, far below the gap of two keys.
__device__ void router_phase(const FewArgs& a) {
    const int lane = threadIdx.x & 31;
    const int nch = a.H / 8;
    const int per = (nch + a.n_split - 1) / a.n_split;
    const int units = a.E * a.n_split;
    for (int u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
        const int e = u / a.n_split, sp = u % a.n_split;
        const int c1 = min(nch, (sp + 1) * per);
        const uint4* wr = reinterpret_cast<const uint4*>(a.w_router + (size_t)e * a.H);
        for (int t = 0; t < a.T; ++t) {
            const uint4* xr = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H);
            double acc = 0.0;
#pragma unroll 4
            for (int c = sp * per + lane; c < c1; c += 32) {
                float w[8], x[8], s = 0.0f;
                unpack8(__ldg(wr + c), w);
                unpack8(__ldg(xr + c), x);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(w[j], x[j], s);
                acc += (double)s;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
            if (lane == 0) a.part[((size_t)sp * a.T + t) * a.E + e] = acc;
        }
    }
}

// The choice of token t by one warp; `key` holds E values.
__device__ void choose(const FewArgs& a, int t, double* key, Plan* P) {
    const int lane = threadIdx.x & 31;
    for (int e = lane; e < a.E; e += 32) {
        double l = 0.0;
        for (int sp = 0; sp < a.n_split; ++sp) l += __ldcg(a.part + ((size_t)sp * a.T + t) * a.E + e);
        const double c = 1.0 / (1.0 + exp(-l)) + (double)__ldg(a.bias + e);
        key[e] = isnan(c) ? -INFINITY : c;   // NaN ranks below numbers
    }
    __syncwarp();
    uint32_t keep = 0xffffffffu;
    const int gsz = a.E / a.n_group;
    if (a.n_group > 1) {
        // lane g: the sum of group g's group_topn largest keys, largest first
        double gs = -INFINITY;
        if (lane < a.n_group) {
            double lv = INFINITY;
            int li = -1;
            for (int j = 0; j < a.group_topn; ++j) {
                double bv = -INFINITY;
                int bi = 0x7fffffff;
                for (int e = lane * gsz; e < (lane + 1) * gsz; ++e)
                    if (better(lv, li, key[e], e) && better(key[e], e, bv, bi)) {
                        bv = key[e];
                        bi = e;
                    }
                gs = j == 0 ? bv : gs + bv;
                lv = bv;
                li = bi;
            }
            if (isnan(gs)) gs = -INFINITY;
        }
        keep = 0;
        bool taken = lane >= a.n_group;
        for (int j = 0; j < a.topk_group; ++j) {
            double bv = taken ? -INFINITY : gs;
            int bi = taken ? 0x7fffffff : lane;
            warp_best(bv, bi);
            keep |= 1u << (bi & 31);
            if (lane == bi) taken = true;
        }
    }
    double my_s = 0.0;
    int my_e = 0;
    double lv = INFINITY;
    int li = -1;
    for (int j = 0; j < a.k; ++j) {
        double bv = -INFINITY;
        int bi = 0x7fffffff;
        for (int e = lane; e < a.E; e += 32)
            if ((keep >> (a.n_group > 1 ? e / gsz : 0) & 1u) && better(lv, li, key[e], e) &&
                better(key[e], e, bv, bi)) {
                bv = key[e];
                bi = e;
            }
        warp_best(bv, bi);
        lv = bv;
        li = bi;
        if (lane == j) my_e = bi;
    }
    if (lane < a.k) {
        double l = 0.0;
        for (int sp = 0; sp < a.n_split; ++sp) l += __ldcg(a.part + ((size_t)sp * a.T + t) * a.E + my_e);
        my_s = 1.0 / (1.0 + exp(-l));
    }
    double sum = 0.0;
    for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, my_s, j);
    if (lane < a.k) {
        const float w = (float)((a.norm ? my_s / sum : my_s) * (double)a.rsf);
        P->sel[t * a.k + lane] = my_e;
        P->selw[t * a.k + lane] = w;
        if (blockIdx.x == 0) {
            if (a.idx) a.idx[(size_t)t * a.k + lane] = my_e;
            if (a.w) a.w[(size_t)t * a.k + lane] = w;
        }
    }
}

// Touched experts in ascending order after the shared one, with their tokens
// and pairs, from the choice.  All threads.
__device__ void build_plan(const FewArgs& a, Plan* P) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < a.E; e += kThreads) P->emask[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.T * a.k; i += kThreads) atomicOr(&P->emask[P->sel[i]], 1u << (i / a.k));
    __syncthreads();
    if (tid < 32) {
        int n = 0, pairs = 0;
        if (a.Is) {
            if (lane == 0) {
                P->expert[0] = -1;
                P->mask[0] = (1u << a.T) - 1u;
                P->base[0] = 0;
            }
            n = 1;
            pairs = a.T;
        }
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const uint32_t m = P->emask[e0 + lane];
            const int cnt = __popc(m);
            const uint32_t hit = __ballot_sync(0xffffffffu, cnt > 0);
            int incl = cnt;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += v;
            }
            if (cnt) {
                const int p = n + __popc(hit & ((1u << lane) - 1u));
                P->expert[p] = e0 + lane;
                P->mask[p] = m;
                P->base[p] = pairs + incl - cnt;
                P->apos[e0 + lane] = p;
            }
            n += __popc(hit);
            pairs += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) P->n_active = n;
    }
    __syncthreads();
    if (a.Is)
        for (int t = tid; t < a.T; t += kThreads) P->w[t] = 1.0f;
    for (int i = tid; i < a.T * a.k; i += kThreads) {
        const int p = P->apos[P->sel[i]], t = i / a.k;
        P->w[P->base[p] + __popc(P->mask[p] & ((1u << t) - 1u))] = P->selw[i];
    }
    __syncthreads();
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Plan* P = reinterpret_cast<Plan*>(smem);
    double* keys = reinterpret_cast<double*>(smem + (sizeof(Plan) + 15) / 16 * 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) P->abort = 0;
    router_phase(a);
    if (!grid_barrier(a, 0, &P->abort)) return;
    for (int t = warp; t < a.T; t += kWarps) choose(a, t, keys + warp * a.E, P);
    __syncthreads();
    build_plan(a, P);

    // phase 1: a warp per (expert, SwiGLU feature)
    const int nwarp = gridDim.x * kWarps, gw = blockIdx.x * kWarps + warp;
    int first = 0;
    for (int p = 0; p < P->n_active; ++p) {
        const int e = P->expert[p];
        const int n = e < 0 ? a.Is : a.I;
        const uint8_t* w = e < 0 ? a.w13s : a.w13;
        const void* s = e < 0 ? a.s13s : a.s13;
        const size_t row0 = e < 0 ? 0 : (size_t)e * 2 * a.I;
        for (int f = (gw + nwarp - first % nwarp) % nwarp; f < n; f += nwarp) {
            int pair = P->base[p];
            for (uint32_t m = P->mask[p]; m; m &= m - 1, ++pair) {
                const uint16_t* xr = a.x + (size_t)(__ffs(m) - 1) * a.H;
                float g = 0.0f, u = 0.0f;
                for (int k = lane * 8; k < a.H; k += 256) {
                    float x[8], wg[8], wu[8];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(xr + k)), x);
                    load8<DT>(w, s, row0 + f, a.H, k, wg);
                    load8<DT>(w, s, row0 + n + f, a.H, k, wu);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        g = fmaf(wg[j], x[j], g);
                        u = fmaf(wu[j], x[j], u);
                    }
                }
                g = warp_sum(g);
                u = warp_sum(u);
                if (lane == 0)
                    a.act[(size_t)pair * a.ld_act + f] = g / (1.0f + expf(-g)) * u * P->w[pair];
            }
        }
        first += n;
    }
    if (!grid_barrier(a, 1, &P->abort)) return;

    // phase 2: a warp per output feature
    for (int h = gw; h < a.H; h += nwarp) {
        float acc[kT];
#pragma unroll
        for (int t = 0; t < kT; ++t) acc[t] = 0.0f;
        for (int p = 0; p < P->n_active; ++p) {
            const int e = P->expert[p];
            const int n = e < 0 ? a.Is : a.I;
            const uint8_t* w = e < 0 ? a.w2s : a.w2;
            const void* s = e < 0 ? a.s2s : a.s2;
            const size_t row = (e < 0 ? 0 : (size_t)e * a.H) + h;
            for (int k = lane * 8; k < n; k += 256) {
                float wd[8];
                load8<DT>(w, s, row, n, k, wd);
                int pair = P->base[p];
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    if (!(P->mask[p] >> t & 1u)) continue;
                    const float* ar = a.act + (size_t)pair++ * a.ld_act + k;
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[t] = fmaf(wd[j], __ldcg(ar + j), acc[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const float v = warp_sum(acc[t]);
            if (lane == 0 && t < a.T) {
                const __nv_bfloat16 b = __float2bfloat16_rn(v);
                a.out[(size_t)t * a.H + h] = *reinterpret_cast<const uint16_t*>(&b);
            }
        }
    }
    // the last block to leave clears the counters for the next launch
    if (threadIdx.x == 0) {
        int* bar = a.status + kBarWord;
        if (atomicAdd(bar + 2, 1) == (int)gridDim.x - 1) {
            bar[0] = 0;
            bar[1] = 0;
            bar[2] = 0;
        }
    }
}

// ------------------------------------------------------------------ host side
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct FewLayout {
    size_t part, act, total;
    int n_split, ld_act;
};

// K slices of the router: enough that every warp of the grid has one.
FewLayout few_layout(const moe_config_t* c) {
    FewLayout L{};
    const int nch = c->H / 256 > 0 ? c->H / 256 : 1;
    int split = 148 * kWarps / c->E;
    split = split < 1 ? 1 : split > nch ? nch : split;
    L.n_split = split;
    const int Is = c->n_shared * c->I;
    L.ld_act = Is > c->I ? Is : c->I;
    size_t off = 256;
    L.part = off;
    off += up256((size_t)split * c->T * c->E * 8);
    L.act = off;
    off += up256((size_t)c->T * (c->k + 1) * L.ld_act * 4);
    L.total = off;
    return L;
}

moe_status_t ffail(moe_status_t st, const char* fmt, const char* a, long long b = 0, long long c = 0) {
    char msg[256];
    snprintf(msg, sizeof(msg), fmt, a, b, c);
    return moe::api_fail(st, msg);
}

#define FEW_TRY(x)                         \
    do {                                   \
        moe_status_t st_ = (x);            \
        if (st_ != MOE_OK) return st_;     \
    } while (0)

moe_status_t need(const void* p, const char* name, size_t align) {
    if (!p) return ffail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return ffail(MOE_ERR_INVALID_ARG, "%s must be %lld-byte aligned", name, (long long)align);
    return MOE_OK;
}

moe_status_t few_check(const moe_config_t* c) {
    if (!c) return moe::api_fail(MOE_ERR_INVALID_ARG, "config is NULL");
    moe_config_t b = *c;
    if (b.dtype == MOE_DTYPE_MXFP4_BLOCK32) b.dtype = MOE_DTYPE_BF16;
    FEW_TRY(moe::api_check_config(&b));
    if (c->T > kT)
        return ffail(MOE_ERR_UNSUPPORTED, "%s=%lld is above %lld: use moe_forward", "T", c->T, kT);
    return MOE_OK;
}

template <int DT>
moe_status_t launch_few(FewArgs& a, cudaStream_t s) {
    const size_t smem = (sizeof(Plan) + 15) / 16 * 16 + (size_t)kWarps * a.E * 8;
    int sms = 0;
    FEW_TRY(moe::api_sm_count(&sms));
    cudaError_t e = cudaFuncSetAttribute(few_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) {
        void* args[] = {&a};
        e = cudaLaunchCooperativeKernel(few_kernel<DT>, dim3(sms), dim3(kThreads), args, smem, s);
    }
    if (e != cudaSuccess) return ffail(MOE_ERR_CUDA, "few-token layer launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_few_workspace_size(const moe_config_t* cfg) {
    moe::api_clear_error();
    if (few_check(cfg) != MOE_OK) return 0;
    return few_layout(cfg).total;
}

moe_status_t moe_forward_few(const moe_config_t* cfg, const void* x, const void* w_router,
                             const float* bias, const void* w13, const void* w13_scale,
                             const void* w2, const void* w2_scale, const void* w13s,
                             const void* w13s_scale, const void* w2s, const void* w2s_scale,
                             void* out, int32_t* topk_idx, float* topk_w, void* ws,
                             size_t ws_bytes, moe_stream_t stream) {
    moe::api_clear_error();
    FEW_TRY(few_check(cfg));
    if (cfg->T == 0) return MOE_OK;
    FEW_TRY(need(x, "x", 16));
    FEW_TRY(need(w_router, "w_router", 16));
    FEW_TRY(need(bias, "bias", 4));
    FEW_TRY(need(w13, "w13", 16));
    FEW_TRY(need(w2, "w2", 16));
    FEW_TRY(need(out, "out", 16));
    if (topk_idx) FEW_TRY(need(topk_idx, "topk_idx", 4));
    if (topk_w) FEW_TRY(need(topk_w, "topk_w", 4));
    const bool shared = cfg->n_shared > 0;
    if (shared) {
        FEW_TRY(need(w13s, "w13s", 16));
        FEW_TRY(need(w2s, "w2s", 16));
    }
    if (cfg->dtype == MOE_DTYPE_BF16) {
        if (w13_scale || w2_scale || w13s_scale || w2s_scale)
            return moe::api_fail(MOE_ERR_INVALID_ARG, "weight scales given for bf16 weights");
    } else {
        const size_t al = cfg->dtype == MOE_DTYPE_MXFP4_BLOCK32 ? 16 : 4;
        FEW_TRY(need(w13_scale, "w13_scale", al));
        FEW_TRY(need(w2_scale, "w2_scale", al));
        if (shared) {
            FEW_TRY(need(w13s_scale, "w13s_scale", al));
            FEW_TRY(need(w2s_scale, "w2s_scale", al));
        }
    }
    FEW_TRY(need(ws, "workspace", 256));
    const FewLayout L = few_layout(cfg);
    if (ws_bytes < L.total)
        return ffail(MOE_ERR_WORKSPACE, "workspace has too few bytes, %s %lld", "needs", (long long)L.total);
    FewArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.w_router = static_cast<const uint16_t*>(w_router);
    a.bias = bias;
    a.w13 = static_cast<const uint8_t*>(w13);
    a.w2 = static_cast<const uint8_t*>(w2);
    a.w13s = static_cast<const uint8_t*>(w13s);
    a.w2s = static_cast<const uint8_t*>(w2s);
    a.s13 = w13_scale;
    a.s2 = w2_scale;
    a.s13s = w13s_scale;
    a.s2s = w2s_scale;
    a.out = static_cast<uint16_t*>(out);
    a.idx = topk_idx;
    a.w = topk_w;
    char* base = static_cast<char*>(ws);
    a.status = reinterpret_cast<int*>(base);
    a.part = reinterpret_cast<double*>(base + L.part);
    a.act = reinterpret_cast<float*>(base + L.act);
    a.T = cfg->T;
    a.H = cfg->H;
    a.E = cfg->E;
    a.k = cfg->k;
    a.I = cfg->I;
    a.Is = cfg->n_shared * cfg->I;
    a.n_group = cfg->n_group;
    a.topk_group = cfg->topk_group;
    a.group_topn = cfg->group_topn;
    a.norm = cfg->norm_topk_prob != 0;
    a.rsf = cfg->routed_scaling_factor;
    a.n_split = L.n_split;
    a.ld_act = L.ld_act;
    a.stall = cfg->flags & MOE_FLAG_TEST_STALL ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (cfg->dtype) {
        case MOE_DTYPE_BF16: return launch_few<MOE_DTYPE_BF16>(a, s);
        case MOE_DTYPE_FP8_E4M3_BLOCK128: return launch_few<MOE_DTYPE_FP8_E4M3_BLOCK128>(a, s);
        default: return launch_few<MOE_DTYPE_MXFP4_BLOCK32>(a, s);
    }
}

}  // extern "C"
