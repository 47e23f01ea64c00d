// few.cu -- the whole MoE FFN layer for a few tokens in one launch
// (moe_forward_few): router, choice, the experts' SwiGLU and the combine.
//
// Steps a1-a9 of the layer (sources in include/moe.h).  With 1..16 tokens the
// weights of the touched experts are all the traffic and every one is used a
// handful of times, so the kernel is a weight stream: one cooperative launch,
// one block per SM, each block walking its share of the weight rows through a
// shared-memory ring while the multiplications keep up behind it.
//
// Roles in a block (17 warps):
//   warp 16     producer: bulk copies of weight rows and of the activations
//               they meet, stage by stage, as far ahead as the ring is deep
//   warps 0-7   consumers: m16n8k16 matrix instructions, 16 weight rows by 8
//               tokens; the tokens are the short side, so the 128-row tiles
//               of tcgen05 would be coarse units to share out over 148 SMs
//               (a decode token touches 1728 16-row units but 216 of 128
//               rows), and 4- and 8-bit weights need their values widened in
//               registers anyway
//   warps 8-15  router: logits, choice and the plan of touched experts, while
//               the consumers already work on the shared expert, which needs
//               no choice
//
// Phases:
//   R   a warp per (expert, K slice) of the logits; grid barrier 0; then every
//       block repeats the choice (T * E keys) and the plan
//   1   units of nf SwiGLU features of one expert (nf gate rows, nf up rows,
//       all of K): SiLU(g) * u * w leaves as a bf16 head and a bf16 tail (16
//       significand bits) in the workspace; grid barrier 1
//   2   the output rows' sum over all (expert, k) as one long K axis, shared
//       out evenly to 128 columns; a row block that two or more blocks share
//       is joined by the last of them, in block order
// The producer issues phase 2's weight copies without waiting for barrier 1;
// only the copies of the activations wait for it.
//
// 8- and 4-bit weights become bf16 by moving their bits into a bf16's sign,
// exponent and mantissa fields (e4m3 as value * 2^-120, e2m1 as value *
// 2^-126: subnormals stay subnormals, so no case is special); the activations
// carry 2^64, and the products are brought back (2^56, 2^62) together with the
// block scales, in fp32.  Nothing is rounded on the way.
#include "moe.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

#include <cuda_bf16.h>
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
constexpr int kWarps = 8;                        // consumers, and as many router warps
constexpr int kGroup = kWarps * 32;
constexpr int kThreads = 2 * kGroup + 32;
constexpr int kChunk = 512;                      // K columns of a full stage
constexpr int kXStride = kChunk * 2 + 64;        // bytes between activation rows of a stage
constexpr int kXStrideHalf = kChunk + 64;        // the same of a 256-column stage
constexpr int kMaxStages = 16;
constexpr int kBarWord = moe::kSchedFirstWord;   // grid barriers (2) and the exit count, in the status block
constexpr float kLift = 0x1p64f;                 // factor of the activations for 8- and 4-bit weights

// Per weight type: rows of a unit, smem bytes between rows, bits per weight.
// A stage holds about 17 KB of weights.  Row strides keep a fragment load's
// lanes (8 rows x 4 lanes of 16, 8 or 4 bytes) on different banks.
template <int DT>
struct Fmt;
template <>
struct Fmt<MOE_DTYPE_BF16> {
    static constexpr int kRows = 16, kStride = 1024 + 64, kBits = 16, kScaleStride = 0;
};
template <>
struct Fmt<MOE_DTYPE_FP8_E4M3_BLOCK128> {
    static constexpr int kRows = 32, kStride = 512 + 32, kBits = 8, kScaleStride = 0;
};
template <>
struct Fmt<MOE_DTYPE_MXFP4_BLOCK32> {
    static constexpr int kRows = 64, kStride = 256 + 16, kBits = 4, kScaleStride = 32;
};

struct FewArgs {
    const uint16_t *x, *w_router;
    const float* bias;
    const uint8_t *w13, *w2, *w13s, *w2s;
    const void *s13, *s2, *s13s, *s2s;
    uint16_t* out;
    int32_t* idx;
    float* w;
    int* status;
    double* part;               // [n_split][T][E] logits of the K slices
    uint16_t *act_hi, *act_lo;  // [pairs][ld_act] weighted SwiGLU outputs, head and tail
    float* join;                // [blocks][2][T][rows] partial sums of shared row blocks
    int* joined;                // [row blocks] blocks that have left theirs
    int T, H, E, k, I, Is, n_group, topk_group, group_topn, norm, n_split, stall, ld_act;
    float rsf;
    // shared-memory layout (bytes)
    int off_active, off_pairw, off_scratch, off_ring, stage_bytes, off_x, n_stages;
};

// One touched expert: its tokens (bit mask), their number and its first
// (expert, token) pair.  expert -1 is the shared one.
struct Active {
    int expert;
    uint32_t mask;
    int base, count;
};

// The plan, the same in every block.
struct Plan {
    Active* active;
    float* pairw;      // routing weight of a pair
    int* n_active;
};

// Scratch of the router warps; the consumers' reduction buffer is apart.
struct Scratch {
    double* keys;      // [min(T, 8)][E]
    int* sel;          // [T, k]
    float* selw;       // [T, k]
    uint32_t* emask;   // [E] tokens of each expert
    int* apos;         // [E] its place in the list
};

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Barrier of the `kGroup` threads of a role; true when any of them says `bad`.
__device__ __forceinline__ bool group_any(int id, bool bad) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)bad), "r"(kGroup)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Untiled bulk copy global -> shared (both 16-byte aligned, bytes a multiple
// of 16), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                               uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// e8m0 scale byte -> binary32 (0 is 2^-127, 255 NaN)
__device__ __forceinline__ float e8m0(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
}

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

// Phase R: logits of expert e over one K slice, one warp each.  Eight exact
// products are summed in binary32, those sums in binary64: the logit's error
// stays near 2^-25 of a partial sum, far below the gap of two keys.
__device__ void router_phase(const FewArgs& a, int warp) {
    const int lane = threadIdx.x & 31;
    const int nch = a.H / 8;
    const int per = (nch + a.n_split - 1) / a.n_split;
    const int units = a.E * a.n_split;
    for (int u = blockIdx.x * kWarps + warp; u < units; u += gridDim.x * kWarps) {
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
__device__ void choose(const FewArgs& a, int t, double* key, const Scratch& S) {
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
        S.sel[t * a.k + lane] = my_e;
        S.selw[t * a.k + lane] = w;
        if (blockIdx.x == 0) {
            if (a.idx) a.idx[(size_t)t * a.k + lane] = my_e;
            if (a.w) a.w[(size_t)t * a.k + lane] = w;
        }
    }
}

// Touched experts in ascending order after the shared one, with their tokens
// and pairs, from the choice.  All router threads; `tid` within them.
__device__ void build_plan(const FewArgs& a, const Plan& P, const Scratch& S, int tid) {
    const int lane = tid & 31;
    for (int e = tid; e < a.E; e += kGroup) S.emask[e] = 0;
    group_any(2, false);
    for (int i = tid; i < a.T * a.k; i += kGroup) atomicOr(&S.emask[S.sel[i]], 1u << (i / a.k));
    group_any(2, false);
    if (tid < 32) {
        int n = 0, pairs = 0;
        if (a.Is) {
            if (lane == 0) P.active[0] = Active{-1, (1u << a.T) - 1u, 0, a.T};
            n = 1;
            pairs = a.T;
        }
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const uint32_t m = S.emask[e0 + lane];
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
                P.active[p] = Active{e0 + lane, m, pairs + incl - cnt, cnt};
                S.apos[e0 + lane] = p;
            }
            n += __popc(hit);
            pairs += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) *P.n_active = n;
    }
    group_any(2, false);
    if (a.Is)
        for (int t = tid; t < a.T; t += kGroup) P.pairw[t] = 1.0f;
    for (int i = tid; i < a.T * a.k; i += kGroup) {
        const Active act = P.active[S.apos[S.sel[i]]];
        const int t = i / a.k;
        P.pairw[act.base + __popc(act.mask & ((1u << t) - 1u))] = S.selw[i];
    }
}

// ------------------------------------------------------------------ shares
// What block c of G works on.  Phase 1 units: the shared expert's (known
// before the choice) and the routed experts', each cut into G contiguous
// runs; phase 2: the (row block, expert, K) axis in steps of 128 columns.
// Every step and every H / 128 of a unit move the same bytes, so phase 2's
// cuts make up for what phase 1's whole units leave uneven.
struct Shares {
    int G, us, ur, ublk;        // blocks; phase-1 units, shared and routed; steps of a unit
    int ws, wi, wsum, nrb;      // steps of the shared and of a routed expert, of a row block; row blocks
    bool joint1, joint2;        // cuts of the routed units / of phase 2 take earlier ones into account
    long long tot2;

    __device__ int s_at(int c) const { return (int)((long long)c * us / G); }
    __device__ int r_at(int c) const {
        return joint1 ? (int)((long long)c * (us + ur) / G) - s_at(c) : (int)((long long)c * ur / G);
    }
    __device__ long long b_at(int c) const {
        if (!joint2) return c * tot2 / G;
        const long long tot = (long long)(us + ur) * ublk + tot2;
        return c * tot / G - (long long)(s_at(c) + r_at(c)) * ublk;
    }
};

template <int DT>
__device__ Shares make_shares(const FewArgs& a, int n_active) {
    constexpr int R = Fmt<DT>::kRows;
    Shares s;
    const int routed = n_active - (a.Is ? 1 : 0);
    s.G = gridDim.x;
    s.us = a.Is / (R / 2);
    s.ur = routed * (a.I / (R / 2));
    s.ublk = a.H / 128;
    s.ws = a.Is / 128;
    s.wi = a.I / 128;
    s.wsum = s.ws + routed * s.wi;
    s.nrb = a.H / R;
    s.tot2 = (long long)s.nrb * s.wsum;
    // both need every block's earlier part to fit under its even share of the
    // whole, or the cuts would run backwards
    s.joint1 = (s.us + s.ur) / s.G >= (s.us + s.G - 1) / s.G;
    const int most = s.joint1 ? (s.us + s.ur + s.G - 1) / s.G
                              : (s.us + s.G - 1) / s.G + (s.ur + s.G - 1) / s.G;
    s.joint2 = ((long long)(s.us + s.ur) * s.ublk + s.tot2) / s.G >= (long long)most * s.ublk;
    return s;
}

// ------------------------------------------------------------------ the ring
struct Ring {
    uint64_t *full, *empty;
    uint8_t* base;
    int n, slot;
    uint32_t phase;
    __device__ void next() {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// What a stage multiplies: `rows` weight rows of one matrix, columns k0 ..
// k0 + kn - 1, with the activations of `count` pairs.
struct Item {
    int expert;        // -1: shared
    int first;         // first feature (phase 1) or output row (phase 2)
    int n, K;          // features of the expert; K of the matrix
    uint32_t mask;
    int base, count;
    int k0, kn;
};

// Columns of a stage: phase 2 keeps head and tail rows of every pair, and
// above eight pairs they only fit with half the columns.
__device__ __forceinline__ int chunk_cols(bool down, int count) {
    return down && count > 8 ? kChunk / 2 : kChunk;
}
__device__ __forceinline__ int x_stride(bool down, int count) {
    return down && count > 8 ? kXStrideHalf : kXStride;
}

template <int DT>
__device__ __forceinline__ size_t weight_row(const Item& it, bool down, int H, int I, int r) {
    if (down) return (it.expert < 0 ? 0 : (size_t)it.expert * H) + it.first + r;
    // 8 gate rows, then the 8 up rows of the same features, for each 16 rows
    const int f = it.first + (r >> 4) * 8 + (r & 7) + (r & 8 ? it.n : 0);
    return (it.expert < 0 ? 0 : (size_t)it.expert * 2 * I) + f;
}

// Producer, all lanes: the stage's weight rows (and MXFP4 scales).
template <int DT>
__device__ void issue_weights(const FewArgs& a, const Item& it, bool down, const Ring& ring, uint64_t policy) {
    using F = Fmt<DT>;
    const int lane = threadIdx.x & 31;
    const uint8_t* w = down ? (it.expert < 0 ? a.w2s : a.w2) : (it.expert < 0 ? a.w13s : a.w13);
    const uint8_t* sc = static_cast<const uint8_t*>(down ? (it.expert < 0 ? a.s2s : a.s2)
                                                         : (it.expert < 0 ? a.s13s : a.s13));
    const uint32_t bar = moe::smem_addr(&ring.full[ring.slot]);
    const uint32_t dst = moe::smem_addr(ring.base + ring.slot * a.stage_bytes);
    const uint32_t bytes = (uint32_t)it.kn * F::kBits / 8;
    uint32_t total = F::kRows * bytes + (uint32_t)it.count * (down ? 2 : 1) * it.kn * 2;
    if (F::kScaleStride) {
        // a row's scales start at any multiple of 4 bytes: copy the 16-byte
        // window around them (a matrix is a multiple of 128 rows, so the
        // window never leaves it)
        uint32_t len = 0;
        for (int r = lane; r < F::kRows; r += 32) {
            const size_t at = (weight_row<DT>(it, down, a.H, a.I, r) * it.K + it.k0) / 32;
            len += (uint32_t)(((at + it.kn / 32 + 15) & ~(size_t)15) - (at & ~(size_t)15));
        }
        total += __reduce_add_sync(0xffffffffu, len);
    }
    if (lane == 0) moe::mbar_arrive_expect_tx(&ring.full[ring.slot], total);
    __syncwarp();
    for (int r = lane; r < F::kRows; r += 32) {
        const size_t at = weight_row<DT>(it, down, a.H, a.I, r) * it.K + it.k0;
        bulk_load_hint(dst + r * F::kStride, w + at * F::kBits / 8, bytes, bar, policy);
        if (F::kScaleStride) {
            const size_t s0 = (at / 32) & ~(size_t)15, s1 = (at / 32 + it.kn / 32 + 15) & ~(size_t)15;
            bulk_load(dst + F::kRows * F::kStride + r * F::kScaleStride, sc + s0, (uint32_t)(s1 - s0), bar);
        }
    }
}

// Producer, all lanes: the activation rows of the stage in `slot`.
__device__ void issue_acts(const FewArgs& a, bool down, uint32_t mask, int base, int count, int k0, int kn,
                           const Ring& ring, int slot) {
    const int lane = threadIdx.x & 31;
    const uint32_t bar = moe::smem_addr(&ring.full[slot]);
    const uint32_t dst = moe::smem_addr(ring.base + slot * a.stage_bytes + a.off_x);
    if (down) {
        if (lane < 2 * count) {
            const int i = lane < count ? lane : lane - count;
            const uint16_t* src = (lane < count ? a.act_hi : a.act_lo) + (size_t)(base + i) * a.ld_act + k0;
            bulk_load(dst + lane * x_stride(true, count), src, kn * 2, bar);
        }
    } else if (mask >> lane & 1u) {
        const int i = __popc(mask & ((1u << lane) - 1u));
        bulk_load(dst + i * kXStride, a.x + (size_t)lane * a.H + k0, kn * 2, bar);
    }
}

// ------------------------------------------------------------------ multiplication
// bf16 pairs of the lane's 8 weights (k = 8 t .. 8 t + 7 of a 32-column
// chunk), in the order the activations' words are put in by order_acts.
__device__ __forceinline__ uint32_t merge_sign(uint32_t sign, uint32_t mag) {
    return (sign & 0x80008000u) | mag;
}
template <int DT>
struct Frag;
template <>
struct Frag<MOE_DTYPE_BF16> {
    uint32_t r[4];
    __device__ __forceinline__ void load(const uint8_t* row, int k) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + k * 2);
        r[0] = v.x;
        r[1] = v.y;
        r[2] = v.z;
        r[3] = v.w;
    }
    __device__ __forceinline__ uint32_t top() const { return 0; }
};
template <>
struct Frag<MOE_DTYPE_FP8_E4M3_BLOCK128> {
    uint32_t r[4], m[4];
    // pairs (0, 2), (1, 3), (4, 6), (5, 7)
    __device__ __forceinline__ void load(const uint8_t* row, int k) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + k);
        const uint32_t c[2] = {v.x, v.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[2 * i] = (c[i] << 4) & 0x07f007f0u;
            m[2 * i + 1] = (c[i] >> 4) & 0x07f007f0u;
            r[2 * i] = merge_sign(c[i] << 8, m[2 * i]);
            r[2 * i + 1] = merge_sign(c[i], m[2 * i + 1]);
        }
    }
    // the largest magnitude field: 0x7f0 is e4m3's NaN
    __device__ __forceinline__ uint32_t top() const {
        return __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
    }
};
template <>
struct Frag<MOE_DTYPE_MXFP4_BLOCK32> {
    uint32_t r[4];
    // pairs (0, 4), (1, 5), (2, 6), (3, 7)
    __device__ __forceinline__ void load(const uint8_t* row, int k) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(row + k / 2);
        r[0] = merge_sign(v << 12, (v << 6) & 0x01c001c0u);
        r[1] = merge_sign(v << 8, (v << 2) & 0x01c001c0u);
        r[2] = merge_sign(v << 4, (v >> 2) & 0x01c001c0u);
        r[3] = merge_sign(v, (v >> 6) & 0x01c001c0u);
    }
    __device__ __forceinline__ uint32_t top() const { return 0; }
};

template <int DT>
__device__ __forceinline__ void order_acts(uint4& b) {
    uint4 o;
    if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
        o.x = __byte_perm(b.x, b.y, 0x5410);
        o.y = __byte_perm(b.x, b.y, 0x7632);
        o.z = __byte_perm(b.z, b.w, 0x5410);
        o.w = __byte_perm(b.z, b.w, 0x7632);
        b = o;
    } else if (DT == MOE_DTYPE_MXFP4_BLOCK32) {
        o.x = __byte_perm(b.x, b.z, 0x5410);
        o.y = __byte_perm(b.x, b.z, 0x7632);
        o.z = __byte_perm(b.y, b.w, 0x5410);
        o.w = __byte_perm(b.y, b.w, 0x7632);
        b = o;
    }
}
__device__ __forceinline__ uint32_t lift2(uint32_t v) {
    const __nv_bfloat162 f = __floats2bfloat162_rn(kLift, kLift);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), f);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// One warp's part of a stage: 16 rows by its K slice, for NT tiles of 8
// columns.  xrow: the stage's activation row of this lane's column, or -1.
// In phase 2 a column is a token, and only the expert's own tokens add the
// stage's products: an infinity or a NaN among its weights reaches no other.
template <int DT, int NT, bool DOWN>
__device__ __forceinline__ void mma_stage(const FewArgs& a, const Item& it, const uint8_t* stage, int mt, int kw,
                                          const int (&xrow)[NT], bool tile1, const float (&fsc)[2][2],
                                          float (&acc)[NT][4]) {
    using F = Fmt<DT>;
    constexpr int KW = kWarps / (F::kRows / 16);
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int per = (it.kn / KW + 31) & ~31;
    const int klo = kw * per, khi = min(it.kn, klo + per);
    const uint8_t* w0 = stage + (mt * 16 + g) * F::kStride;
    const uint8_t* w1 = w0 + 8 * F::kStride;
    const int xs = x_stride(DOWN, it.count);
    const uint8_t* x = stage + a.off_x;
    uint32_t top0 = 0, top1 = 0;
    bool own[NT][2];
    float part[NT][4];      // bf16: the stage's products
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        own[nt][0] = !DOWN || (it.mask >> (8 * nt + 2 * t) & 1u);
        own[nt][1] = !DOWN || (it.mask >> (8 * nt + 2 * t + 1) & 1u);
#pragma unroll
        for (int j = 0; j < 4; ++j) part[nt][j] = 0.0f;
    }
    // MXFP4 scale bytes of the lane's two rows, inside their 16-byte windows
    const uint8_t *s0 = nullptr, *s1 = nullptr;
    if (DT == MOE_DTYPE_MXFP4_BLOCK32) {
        const uint8_t* sb = stage + F::kRows * F::kStride + (mt * 16 + g) * F::kScaleStride;
        const uint32_t r0 = (uint32_t)weight_row<DT>(it, DOWN, a.H, a.I, mt * 16 + g);
        const uint32_t r1 = (uint32_t)weight_row<DT>(it, DOWN, a.H, a.I, mt * 16 + g + 8);
        s0 = sb + ((r0 * (uint32_t)(it.K / 32) + it.k0 / 32) & 15u);
        s1 = sb + 8 * F::kScaleStride + ((r1 * (uint32_t)(it.K / 32) + it.k0 / 32) & 15u);
    }
#pragma unroll 2
    for (int k = klo; k < khi; k += 32) {
        Frag<DT> f0, f1;
        f0.load(w0, k + 8 * t);
        f1.load(w1, k + 8 * t);
        const uint32_t m0[4] = {f0.r[0], f1.r[0], f0.r[1], f1.r[1]};
        const uint32_t m1[4] = {f0.r[2], f1.r[2], f0.r[3], f1.r[3]};
        float sc0 = 1.0f, sc1 = 1.0f;
        if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
            top0 = __vmaxu2(top0, f0.top());
            top1 = __vmaxu2(top1, f1.top());
            const bool second = (it.k0 + k) / 128 != (it.k0 + klo) / 128;
            sc0 = second ? fsc[0][1] : fsc[0][0];
            sc1 = second ? fsc[1][1] : fsc[1][0];
        } else if (DT == MOE_DTYPE_MXFP4_BLOCK32) {
            sc0 = e8m0(s0[k / 32]);
            sc1 = e8m0(s1[k / 32]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt == 1 && !tile1) continue;
            const uint8_t* xr = x + max(xrow[nt], 0) * xs + (k + 8 * t) * 2;
            uint4 b = *reinterpret_cast<const uint4*>(xr);
            uint4 lo = make_uint4(0, 0, 0, 0);
            if (DOWN) {
                lo = *reinterpret_cast<const uint4*>(xr + it.count * xs);
                if (xrow[nt] < 0) b = lo = make_uint4(0, 0, 0, 0);
            }
            order_acts<DT>(b);
            if (DOWN) order_acts<DT>(lo);
            if (DT == MOE_DTYPE_BF16) {
                mma_bf16(part[nt], m0, b.x, b.y);
                mma_bf16(part[nt], m1, b.z, b.w);
                if (DOWN) {
                    mma_bf16(part[nt], m0, lo.x, lo.y);
                    mma_bf16(part[nt], m1, lo.z, lo.w);
                }
            } else {
                if (!DOWN) b = make_uint4(lift2(b.x), lift2(b.y), lift2(b.z), lift2(b.w));
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_bf16(c, m0, b.x, b.y);
                mma_bf16(c, m1, b.z, b.w);
                if (DOWN) {
                    mma_bf16(c, m0, lo.x, lo.y);
                    mma_bf16(c, m1, lo.z, lo.w);
                }
                constexpr float kBack = DT == MOE_DTYPE_MXFP4_BLOCK32 ? 0x1p62f : 0x1p56f;
                if (own[nt][0]) {
                    acc[nt][0] = fmaf(c[0] * kBack, sc0, acc[nt][0]);
                    acc[nt][2] = fmaf(c[2] * kBack, sc1, acc[nt][2]);
                }
                if (own[nt][1]) {
                    acc[nt][1] = fmaf(c[1] * kBack, sc0, acc[nt][1]);
                    acc[nt][3] = fmaf(c[3] * kBack, sc1, acc[nt][3]);
                }
            }
        }
    }
    if (DT == MOE_DTYPE_BF16) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (own[nt][0]) {
                acc[nt][0] += part[nt][0];
                acc[nt][2] += part[nt][2];
            }
            if (own[nt][1]) {
                acc[nt][1] += part[nt][1];
                acc[nt][3] += part[nt][3];
            }
        }
    }
    if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
        // a NaN code anywhere in a row makes its sums NaN
        const uint32_t n0 = __vcmpeq2(top0, 0x07f007f0u), n1 = __vcmpeq2(top1, 0x07f007f0u);
        if (__any_sync(0xffffffffu, n0 | n1)) {
            const float nan = __int_as_float(0x7fc00000);
            const bool r0 = __ballot_sync(0xffffffffu, n0 != 0) >> (lane & 28) & 15u;
            const bool r1 = __ballot_sync(0xffffffffu, n1 != 0) >> (lane & 28) & 15u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (own[nt][j]) {
                        if (r0) acc[nt][j] = nan;
                        if (r1) acc[nt][j + 2] = nan;
                    }
        }
    }
}

// FP8 block scales of a warp's rows and K slice (at most two 128-column
// blocks), fetched before the stage's data is waited for.
template <int DT>
__device__ __forceinline__ void fetch_scales(const FewArgs& a, const Item& it, bool down, int mt, int kw,
                                             float (&fsc)[2][2]) {
    if (DT != MOE_DTYPE_FP8_E4M3_BLOCK128) return;
    constexpr int KW = kWarps / (Fmt<DT>::kRows / 16);
    const float* s = static_cast<const float*>(down ? (it.expert < 0 ? a.s2s : a.s2)
                                                    : (it.expert < 0 ? a.s13s : a.s13));
    const int nb = it.K / 128, per = (it.kn / KW + 31) & ~31;
    const int b0 = min((it.k0 + kw * per) / 128, nb - 1), b1 = min(b0 + 1, nb - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const size_t row = weight_row<DT>(it, down, a.H, a.I, mt * 16 + 8 * i) / 128;
        fsc[i][0] = __ldg(s + row * nb + b0);
        fsc[i][1] = __ldg(s + row * nb + b1);
    }
}

// ------------------------------------------------------------------ the kernel
template <int DT, int NT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
    using F = Fmt<DT>;
    constexpr int R = F::kRows, MT = R / 16, KW = kWarps / MT, NF = R / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], plan_ready;
    __shared__ float4 red[2][kWarps][NT][32];
    __shared__ int n_active_sh, abort_sh, last_sh;
    volatile int* abort_flag = &abort_sh;
    Plan P{reinterpret_cast<Active*>(smem + a.off_active), reinterpret_cast<float*>(smem + a.off_pairw),
           &n_active_sh};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.n_stages; ++i) {
            moe::mbar_init(&full[i], 1);        // the producer's arrive with the stage's bytes
            moe::mbar_init(&empty[i], kWarps);  // one arrive per consumer warp
        }
        moe::mbar_init(&plan_ready, 1);
        abort_sh = 0;
        moe::fence_barrier_init();
    }
    __syncthreads();
    Ring ring{full, empty, smem + a.off_ring, a.n_stages, 0, 0};
    int* bars = a.status + kBarWord;
    const int cta = blockIdx.x;
    const Active shared{-1, (1u << a.T) - 1u, 0, a.T};
    const int first_routed = a.Is ? 1 : 0;

    if (warp >= kWarps && warp < 2 * kWarps) {
        // ---------------------------------------------------------- router
        const int tid = threadIdx.x - kGroup, rw = warp - kWarps;
        Scratch S;
        S.keys = reinterpret_cast<double*>(smem + a.off_scratch);
        S.sel = reinterpret_cast<int*>(S.keys + (size_t)min(a.T, kWarps) * a.E);
        S.selw = reinterpret_cast<float*>(S.sel + a.T * a.k);
        S.emask = reinterpret_cast<uint32_t*>(S.selw + a.T * a.k);
        S.apos = reinterpret_cast<int*>(S.emask + a.E);
        for (int i = cta * kGroup + tid; i < a.H / R; i += gridDim.x * kGroup) a.joined[i] = 0;
        router_phase(a, rw);
        __threadfence();
        group_any(2, false);
        bool ok = true;
        if (tid == 0) {
            if (!(a.stall && cta == 0)) atomicAdd(bars, 1);
            const long long t0 = clock64();
            while (*reinterpret_cast<volatile int*>(bars) < (int)gridDim.x) {
                if (clock64() - t0 > moe::kWaitLimit) {
                    atomicOr(a.status, moe::DEV_STATUS_TIMEOUT);
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
            }
            __threadfence();
        }
        if (!group_any(2, !ok)) {
            for (int t = rw; t < a.T; t += kWarps) choose(a, t, S.keys + (size_t)rw * a.E, S);
            group_any(2, false);
            build_plan(a, P, S, tid);
            group_any(2, false);
            if (tid == 0) moe::mbar_arrive(&plan_ready);
        }
    } else if (warp == 2 * kWarps) {
        // ---------------------------------------------------------- producer
        const uint64_t policy = moe::l2_policy_evict_first();
        bool ok = true;
        uint32_t issued = 0, last_phase = 0;   // slots in use, and their newest phase
        auto claim = [&]() {
            ok = __all_sync(0xffffffffu,
                            moe::wait_bar(&ring.empty[ring.slot], ring.phase ^ 1, abort_flag, a.status));
            return ok;
        };
        auto mark = [&]() {
            issued |= 1u << ring.slot;
            last_phase = (last_phase & ~(1u << ring.slot)) | (ring.phase << ring.slot);
        };
        auto gate_up = [&](const Active& act, int n, int f0) {
            Item it{act.expert, f0, n, a.H, act.mask, act.base, act.count, 0, 0};
            for (; it.k0 < a.H; it.k0 += kChunk) {
                it.kn = min(kChunk, a.H - it.k0);
                if (!claim()) return;
                issue_weights<DT>(a, it, false, ring, policy);
                issue_acts(a, false, it.mask, 0, it.count, it.k0, it.kn, ring, ring.slot);
                mark();
                ring.next();
            }
        };
        Shares sh = make_shares<DT>(a, first_routed);
        for (int u = sh.s_at(cta); ok && u < sh.s_at(cta + 1); ++u) gate_up(shared, a.Is, u * NF);
        if (ok) ok = __all_sync(0xffffffffu, moe::wait_bar(&plan_ready, 0, abort_flag, a.status));
        if (ok) {
            sh = make_shares<DT>(a, n_active_sh);
            const int upe = a.I / NF;
            for (int u = sh.r_at(cta); ok && u < sh.r_at(cta + 1); ++u)
                gate_up(P.active[first_routed + u / upe], a.I, (u % upe) * NF);

            // phase 2: lane i remembers what slot i still lacks
            bool open = false;                 // barrier 1 has been passed
            int lack = 0, l_base = 0, l_count = 0, l_k0 = 0, l_kn = 0;
            auto supply = [&]() {
                fence_proxy_async();           // the heads and tails are other blocks' plain stores
                for (uint32_t m = __ballot_sync(0xffffffffu, lack); m; m &= m - 1) {
                    const int sl = __ffs(m) - 1;
                    issue_acts(a, true, 0, __shfl_sync(0xffffffffu, l_base, sl),
                               __shfl_sync(0xffffffffu, l_count, sl), __shfl_sync(0xffffffffu, l_k0, sl),
                               __shfl_sync(0xffffffffu, l_kn, sl), ring, sl);
                }
                lack = 0;
            };
            auto poll = [&]() {
                int n = 0;
                if (lane == 0) {
                    n = *reinterpret_cast<volatile int*>(bars + 1);
                    __threadfence();
                }
                return __shfl_sync(0xffffffffu, n, 0) >= (int)gridDim.x;
            };
            long long pos = sh.b_at(cta);
            const long long end = sh.b_at(cta + 1);
            long long t0 = clock64();
            while (ok && pos < end) {
                const int rb = (int)(pos / sh.wsum);
                int off = (int)(pos % sh.wsum);
                int p, K;
                if (off < sh.ws) {
                    p = 0;
                    K = a.Is;
                } else {
                    p = first_routed + (off - sh.ws) / sh.wi;
                    off = (off - sh.ws) % sh.wi;
                    K = a.I;
                }
                const Active act = P.active[p];
                const int cols = chunk_cols(true, act.count);
                const int left = (int)min((long long)(K / 128 - off), end - pos) * 128;
                Item it{act.expert, rb * R, 0, K, act.mask, act.base, act.count, off * 128, min(cols, left)};
                // a free slot, or barrier 1 so that the consumers can make one
                while (true) {
                    if (__all_sync(0xffffffffu, moe::mbar_try_wait(&ring.empty[ring.slot], ring.phase ^ 1))) break;
                    if (!open && poll()) {
                        open = true;
                        supply();
                    }
                    bool late = false;
                    if (lane == 0 && (*abort_flag || clock64() - t0 > moe::kWaitLimit)) {
                        if (!*abort_flag) atomicOr(a.status, moe::DEV_STATUS_TIMEOUT);
                        *abort_flag = 1;
                        late = true;
                    }
                    if (__any_sync(0xffffffffu, late)) {
                        ok = false;
                        break;
                    }
                }
                if (!ok) break;
                t0 = clock64();
                issue_weights<DT>(a, it, true, ring, policy);
                mark();
                if (open) {
                    issue_acts(a, true, 0, it.base, it.count, it.k0, it.kn, ring, ring.slot);
                } else if (lane == ring.slot) {
                    lack = 1;
                    l_base = it.base;
                    l_count = it.count;
                    l_k0 = it.k0;
                    l_kn = it.kn;
                }
                ring.next();
                pos += it.kn / 128;
            }
            while (ok && !open) {
                if (poll()) {
                    open = true;
                    break;
                }
                bool late = false;
                if (lane == 0 && (*abort_flag || clock64() - t0 > moe::kWaitLimit)) {
                    if (!*abort_flag) atomicOr(a.status, moe::DEV_STATUS_TIMEOUT);
                    *abort_flag = 1;
                    late = true;
                }
                if (__any_sync(0xffffffffu, late)) ok = false;
            }
            supply();   // also when giving up: every stage's bytes then arrive
        }
        // no copy may still be in flight when the block leaves
        if (!ok)
            for (int i = 0; i < a.n_stages; ++i)
                if (issued >> i & 1u) moe::wait_bar(&full[i], last_phase >> i & 1u, abort_flag, a.status, true);
    } else {
        // ---------------------------------------------------------- consumers
        const int mt = warp / KW, kw = warp % KW, tid = threadIdx.x;
        const int g = lane >> 2, t = lane & 3;
        int buf = 0;
        bool ok = true;
        float acc[NT][4];
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        };
        // one stage; false when the wait was given up
        auto stage_gate_up = [&](const Item& it) {
            int xrow[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) xrow[i] = 8 * i + g < it.count ? 8 * i + g : 0;
            float fsc[2][2] = {};
            fetch_scales<DT>(a, it, false, mt, kw, fsc);
            ok = __all_sync(0xffffffffu, moe::wait_bar(&full[ring.slot], ring.phase, abort_flag, a.status));
            if (!ok) return;
            mma_stage<DT, NT, false>(a, it, ring.base + ring.slot * a.stage_bytes, mt, kw, xrow, it.count > 8, fsc,
                                     acc);
            __syncwarp();
            if (lane == 0) moe::mbar_arrive(&empty[ring.slot]);
            ring.next();
        };
        auto stage_down = [&](const Item& it) {
            int xrow[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int tok = 8 * i + g;
                xrow[i] = it.mask >> tok & 1u ? __popc(it.mask & ((1u << tok) - 1u)) : -1;
            }
            float fsc[2][2] = {};
            fetch_scales<DT>(a, it, true, mt, kw, fsc);
            ok = __all_sync(0xffffffffu, moe::wait_bar(&full[ring.slot], ring.phase, abort_flag, a.status));
            if (!ok) return;
            mma_stage<DT, NT, true>(a, it, ring.base + ring.slot * a.stage_bytes, mt, kw, xrow, it.mask >> 8, fsc,
                                    acc);
            __syncwarp();
            if (lane == 0) moe::mbar_arrive(&empty[ring.slot]);
            ring.next();
        };
        // Leaves the warps' sums in red[buf] and waits for all of them; true
        // when any warp has given up.
        auto gather = [&]() {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                red[buf][warp][i][lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            return group_any(1, !ok);
        };
        // Sum over the K slices: thread tid takes row group tid / (32 NT),
        // column tile (tid / 32) % NT.
        auto reduced = [&]() {
            const int m = tid / (32 * NT), i = tid / 32 % NT;
            float4 s = red[buf][m * KW][i][lane];
#pragma unroll
            for (int q = 1; q < KW; ++q) {
                const float4 v = red[buf][m * KW + q][i][lane];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            return s;
        };
        auto gate_up = [&](const Active& act, int n, int f0) {
            clear();
            Item it{act.expert, f0, n, a.H, act.mask, act.base, act.count, 0, 0};
            for (; ok && it.k0 < a.H; it.k0 += kChunk) {
                it.kn = min(kChunk, a.H - it.k0);
                stage_gate_up(it);
            }
            if (gather()) return false;
            if (tid < MT * NT * 32) {
                const float4 s = reduced();
                const int f = f0 + tid / (32 * NT) * 8 + g, c0 = tid / 32 % NT * 8 + 2 * t;
                const float gate[2] = {s.x, s.y}, up[2] = {s.z, s.w};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (c0 + j >= act.count) continue;
                    const int pair = act.base + c0 + j;
                    float v = gate[j] / (1.0f + expf(-gate[j])) * up[j];
                    if (act.expert >= 0) v *= P.pairw[pair];
                    if (DT != MOE_DTYPE_BF16) v *= kLift;
                    // head and tail: together 16 significand bits
                    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                    const __nv_bfloat16 lo = __float2bfloat16_rn(v - __bfloat162float(hi));
                    const size_t at = (size_t)pair * a.ld_act + f;
                    a.act_hi[at] = *reinterpret_cast<const uint16_t*>(&hi);
                    a.act_lo[at] = *reinterpret_cast<const uint16_t*>(&lo);
                }
            }
            buf ^= 1;
            return true;
        };

        bool good = true;
        Shares sh = make_shares<DT>(a, first_routed);
        for (int u = sh.s_at(cta); good && u < sh.s_at(cta + 1); ++u) good = gate_up(shared, a.Is, u * NF);
        if (good) {
            ok = __all_sync(0xffffffffu, moe::wait_bar(&plan_ready, 0, abort_flag, a.status));
            good = !group_any(1, !ok);
        }
        if (good) {
            sh = make_shares<DT>(a, n_active_sh);
            const int upe = a.I / NF;
            for (int u = sh.r_at(cta); good && u < sh.r_at(cta + 1); ++u)
                good = gate_up(P.active[first_routed + u / upe], a.I, (u % upe) * NF);
        }
        if (good) {
            // barrier 1: this block's heads and tails are written
            __threadfence();
            fence_proxy_async();
            group_any(1, false);
            if (tid == 0) atomicAdd(bars + 1, 1);
            long long pos = sh.b_at(cta);
            const long long begin = pos, end = sh.b_at(cta + 1);
            while (good && pos < end) {
                const int rb = (int)(pos / sh.wsum);
                const long long lo = (long long)rb * sh.wsum, hi = lo + sh.wsum;
                const long long seg0 = pos, seg1 = min(hi, end);
                clear();
                while (ok && pos < seg1) {
                    int off = (int)(pos - lo), p, K;
                    if (off < sh.ws) {
                        p = 0;
                        K = a.Is;
                    } else {
                        p = first_routed + (off - sh.ws) / sh.wi;
                        off = (off - sh.ws) % sh.wi;
                        K = a.I;
                    }
                    const Active act = P.active[p];
                    const int left = (int)min((long long)(K / 128 - off), end - pos) * 128;
                    Item it{act.expert, rb * R, 0, K, act.mask, act.base, act.count, off * 128,
                            min(chunk_cols(true, act.count), left)};
                    stage_down(it);
                    pos += it.kn / 128;
                }
                if (gather()) break;
                const bool whole = seg0 == lo && seg1 == hi;
                float* mine = a.join + ((size_t)cta * 2 + (seg0 == begin ? 0 : 1)) * a.T * R;
                if (tid < MT * NT * 32) {
                    const float4 s = reduced();
                    const int r = tid / (32 * NT) * 16 + g, c0 = tid / 32 % NT * 8 + 2 * t;
                    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int tok = c0 + (j & 1), row = r + (j >> 1) * 8;
                        if (tok >= a.T) continue;
                        if (whole) {
                            const __nv_bfloat16 b = __float2bfloat16_rn(v[j]);
                            a.out[(size_t)tok * a.H + rb * R + row] = *reinterpret_cast<const uint16_t*>(&b);
                        } else {
                            mine[tok * R + row] = v[j];
                        }
                    }
                }
                buf ^= 1;
                if (whole) continue;
                // a row block of several blocks: the last to leave its part
                // adds them up in block order
                int c0 = cta, c1 = cta;
                while (c0 > 0 && sh.b_at(c0) > lo) --c0;
                while (c1 + 1 < sh.G && sh.b_at(c1 + 1) < hi) ++c1;
                int parts = 0;
                for (int c = c0; c <= c1; ++c)
                    parts += min(sh.b_at(c + 1), hi) > max(sh.b_at(c), lo);
                __threadfence();
                group_any(1, false);
                if (tid == 0) {
                    last_sh = atomicAdd(a.joined + rb, 1) == parts - 1;
                    __threadfence();
                }
                group_any(1, false);
                if (last_sh) {
                    for (int i = tid; i < a.T * R; i += kGroup) {
                        float s = 0.0f;
                        for (int c = c0; c <= c1; ++c) {
                            const long long b0 = sh.b_at(c);
                            if (min(sh.b_at(c + 1), hi) <= max(b0, lo)) continue;
                            s += __ldcg(a.join + ((size_t)c * 2 + (b0 >= lo ? 0 : 1)) * a.T * R + i);
                        }
                        const __nv_bfloat16 b = __float2bfloat16_rn(s);
                        a.out[(size_t)(i / R) * a.H + rb * R + i % R] = *reinterpret_cast<const uint16_t*>(&b);
                    }
                }
                group_any(1, false);   // last_sh is read before the next one is written
            }
        }
    }
    __syncthreads();
    // the last block to leave clears the counters for the next launch
    if (threadIdx.x == 0 && atomicAdd(bars + 2, 1) == (int)gridDim.x - 1) {
        bars[0] = 0;
        bars[1] = 0;
        bars[2] = 0;
    }
}

// ------------------------------------------------------------------ host side
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kMaxBlocks = 256;       // blocks the join buffer has room for

struct FewLayout {
    size_t part, hi, lo, join, joined, total;
    int n_split, ld_act;
};

// K slices of the router: enough that every router warp of the grid has one.
FewLayout few_layout(const moe_config_t* c) {
    FewLayout L{};
    const int nch = c->H / 256 > 0 ? c->H / 256 : 1;
    int split = 148 * kWarps / c->E;
    split = split < 1 ? 1 : split > nch ? nch : split;
    L.n_split = split;
    const int Is = c->n_shared * c->I;
    L.ld_act = Is > c->I ? Is : c->I;
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = up256(off + bytes);
        return at;
    };
    L.part = take((size_t)split * c->T * c->E * 8);
    L.hi = take((size_t)c->T * (c->k + 1) * L.ld_act * 2);
    L.lo = take((size_t)c->T * (c->k + 1) * L.ld_act * 2);
    L.join = take((size_t)kMaxBlocks * 2 * c->T * 64 * 4);
    L.joined = take((size_t)c->H / 16 * 4);
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

// Shared memory: plan, router scratch, then as many stages as fit.
template <int DT>
moe_status_t few_smem(FewArgs& a, int limit, size_t* bytes) {
    using F = Fmt<DT>;
    auto up = [](int v, int to) { return (v + to - 1) / to * to; };
    const int n = a.T * a.k, active = (n < a.E ? n : a.E) + 1;
    int off = 0;
    a.off_active = off;
    off += active * (int)sizeof(Active);
    a.off_pairw = off;
    off = up(off + (n + a.T) * 4, 16);
    a.off_scratch = off;
    off += (a.T < kWarps ? a.T : kWarps) * a.E * 8 + n * 8 + a.E * 8;
    a.off_ring = up(off, 128);
    a.off_x = F::kRows * (F::kStride + F::kScaleStride);
    const int x = a.T <= 8 ? 2 * a.T * kXStride : 2 * kT * kXStrideHalf;
    a.stage_bytes = up(a.off_x + x, 128);
    const int stages = (limit - a.off_ring) / a.stage_bytes;
    a.n_stages = stages < kMaxStages ? stages : kMaxStages;
    if (a.n_stages < 2)
        return ffail(MOE_ERR_UNSUPPORTED, "%s: %lld bytes of shared memory hold fewer than two stages", "few-token layer",
                     limit);
    *bytes = (size_t)a.off_ring + (size_t)a.n_stages * a.stage_bytes;
    return MOE_OK;
}

template <int DT, int NT>
moe_status_t launch_few(FewArgs& a, cudaStream_t s) {
    int sms = 0, dev = 0, optin = 0;
    FEW_TRY(moe::api_sm_count(&sms));
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, few_kernel<DT, NT>);
    if (e == cudaSuccess) {
        size_t smem = 0;
        FEW_TRY(few_smem<DT>(a, optin - (int)fa.sharedSizeBytes, &smem));
        e = cudaFuncSetAttribute(few_kernel<DT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) {
            void* args[] = {&a};
            const int grid = sms < kMaxBlocks ? sms : kMaxBlocks;
            e = cudaLaunchCooperativeKernel(few_kernel<DT, NT>, dim3(grid), dim3(kThreads), args, smem, s);
        }
    }
    if (e != cudaSuccess) return ffail(MOE_ERR_CUDA, "few-token layer launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

template <int DT>
moe_status_t launch_tiles(FewArgs& a, cudaStream_t s) {
    return a.T <= 8 ? launch_few<DT, 1>(a, s) : launch_few<DT, 2>(a, s);
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
    a.act_hi = reinterpret_cast<uint16_t*>(base + L.hi);
    a.act_lo = reinterpret_cast<uint16_t*>(base + L.lo);
    a.join = reinterpret_cast<float*>(base + L.join);
    a.joined = reinterpret_cast<int*>(base + L.joined);
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
        case MOE_DTYPE_BF16: return launch_tiles<MOE_DTYPE_BF16>(a, s);
        case MOE_DTYPE_FP8_E4M3_BLOCK128: return launch_tiles<MOE_DTYPE_FP8_E4M3_BLOCK128>(a, s);
        default: return launch_tiles<MOE_DTYPE_MXFP4_BLOCK32>(a, s);
    }
}

}  // extern "C"
