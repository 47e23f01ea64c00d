// few.cu -- the whole MoE FFN layer for a few tokens in one launch
// (moe_forward_few): router, choice, the experts' SwiGLU and the combine.
//
// Steps a1-a9 of the layer (sources in include/moe.h).  With 1..16 tokens the
// weights of the touched experts are all the traffic and every one is used a
// handful of times, so the kernel is a weight stream: one cooperative launch,
// one block per SM, each block walking its share of the weight rows through a
// shared-memory ring while the multiplications keep up behind it.
//
// Roles in a block (13 warps):
//   warp 12     producer: bulk copies of weight rows and of the activations
//               they meet, stage by stage, as far ahead as the ring is deep
//   warps 0-7   consumers: m16n8k16 matrix instructions, 16 weight rows by 8
//               tokens; the tokens are the short side, so the 128-row tiles
//               of tcgen05 would be coarse units to share out over 148 SMs
//               (a decode token touches 1728 16-row units but 216 of 128
//               rows), and 4- and 8-bit weights need their values widened in
//               registers anyway
//   warps 8-11  router: logits, choice and the plan of touched experts, while
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
// 2^-126: subnormals stay subnormals, so no case is special) and one exact
// bf16 product that brings them back; their block scales multiply the products
// in fp32.  Nothing is rounded on the way.
#include "moe.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>

namespace moe {
moe_status_t api_check_config(const moe_config_t* c);
moe_status_t api_fail(moe_status_t st, const char* msg);
void api_clear_error();
moe_status_t api_sm_count(int* n);
moe_status_t api_make_map_u8_sw64(CUtensorMap* m, const void* ptr, uint32_t rank, const uint64_t* dims,
                                  const uint64_t* strides, const uint32_t* box, const char* what);
}  // namespace moe

namespace {

constexpr int kT = MOE_FEW_MAX_T;
constexpr int kWarps = 8;                        // consumers
constexpr int kRouters = 4;
constexpr int kGroup = kWarps * 32, kRouterGroup = kRouters * 32;
constexpr int kThreads = kGroup + kRouterGroup + 32;
constexpr int kChunk = 512;                      // K columns of a full stage
constexpr int kBox = 256;                        // K columns of one tensor copy
constexpr int kBoxBytes = 8192;                  // its bytes, for every weight type
constexpr int kSlice = kChunk / kWarps;          // K columns of a warp in a stage
constexpr int kMaxStages = 16;
constexpr int kBarWord = moe::kSchedFirstWord;   // grid barriers (2) and the exit count, in the status block

// Per weight type: rows of a unit, bits of a weight, bytes of a stage's
// scales, and the activation rows' padding in a stage.  A stage holds 16 KB of
// weights, as 64-byte pieces of 8 rows (512 bytes, 64-byte swizzle): a
// fragment load's lanes (8 rows by four 16-byte pieces) then fall on different
// banks.  The padding does the same for the activations (16 bytes a lane; 32
// for e4m3, whose lanes hold 16 weights).
template <int DT>
struct Fmt;
template <>
struct Fmt<MOE_DTYPE_BF16> {
    static constexpr int kRows = 16, kBits = 16, kScaleBytes = 0, kPad = 64;
};
template <>
struct Fmt<MOE_DTYPE_FP8_E4M3_BLOCK128> {
    static constexpr int kRows = 32, kBits = 8, kScaleBytes = 128, kPad = 16;  // scales: [2][4] fp32
};
template <>
struct Fmt<MOE_DTYPE_MXFP4_BLOCK32> {
    static constexpr int kRows = 64, kBits = 4, kScaleBytes = 1024, kPad = 64;  // [64][16] e8m0
};

struct FewArgs {
    CUtensorMap m13, m2, m13s, m2s;   // weights (see few_maps)
    const uint16_t *x, *w_router;
    const float* bias;
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
    int off_active, off_pairw, off_scratch, off_red, off_ring, stage_bytes, n_stages;
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
    double* keys;      // [min(T, kRouters)][E]
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

// Barrier of the consumers (id 1) or the router warps (id 2); true when any of
// their threads says `bad`.
__device__ __forceinline__ bool group_any(int id, bool bad) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)bad), "r"(id == 1 ? kGroup : kRouterGroup)
        : "memory");
    return r != 0;
}

// Tensor copies of one box, with an L2 policy.
__device__ __forceinline__ void box_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c2, int c3,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void box_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c2, int c4,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %3, %4, %3, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(c2), "r"(c4), "l"(policy)
        : "memory");
}

// Asynchronous copies of 16 or 4 bytes by this thread, and its arrival on
// `bar` once all of them have landed.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_copied(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(moe::smem_addr(bar)) : "memory");
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
    for (int u = blockIdx.x * kRouters + warp; u < units; u += gridDim.x * kRouters) {
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
    for (int e = tid; e < a.E; e += kRouterGroup) S.emask[e] = 0;
    group_any(2, false);
    for (int i = tid; i < a.T * a.k; i += kRouterGroup) atomicOr(&S.emask[S.sel[i]], 1u << (i / a.k));
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
        for (int t = tid; t < a.T; t += kRouterGroup) P.pairw[t] = 1.0f;
    for (int i = tid; i < a.T * a.k; i += kRouterGroup) {
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
    // a cut moves back to the start of its tensor copy (two steps)
    __device__ long long b_at(int c) const {
        long long b;
        if (joint2) {
            const long long tot = (long long)(us + ur) * ublk + tot2;
            b = c * tot / G - (long long)(s_at(c) + r_at(c)) * ublk;
        } else {
            b = c * tot2 / G;
        }
        if (b >= tot2) return tot2;
        const int off = (int)(b % wsum);
        return b - ((off < ws ? off : (off - ws) % wi) & 1);
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
    return down && count > 8 ? kBox : kChunk;
}
template <int DT>
__device__ __forceinline__ int x_stride(int cols) {
    return cols * 2 + Fmt<DT>::kPad;
}
template <int DT>
__host__ __device__ constexpr int off_x() {
    return 2 * kBoxBytes + Fmt<DT>::kScaleBytes;
}

// Row of its matrix that row r of the unit is: phase 1 alternates 8 gate rows
// and the 8 up rows of the same features.
__device__ __forceinline__ size_t weight_row(const Item& it, bool down, int H, int I, int r) {
    if (down) return (it.expert < 0 ? 0 : (size_t)it.expert * H) + it.first + r;
    const int f = it.first + (r >> 4) * 8 + (r & 7) + (r & 8 ? it.n : 0);
    return (it.expert < 0 ? 0 : (size_t)it.expert * 2 * I) + f;
}

// Producer, all lanes: the stage's weights (one tensor copy for each 256
// columns) and scales.
template <int DT>
__device__ void issue_weights(const FewArgs& a, const Item& it, bool down, const Ring& ring, uint64_t policy) {
    using F = Fmt<DT>;
    const int lane = threadIdx.x & 31;
    const uint32_t dst = moe::smem_addr(ring.base + ring.slot * a.stage_bytes);
    if (lane == 0) {
        uint64_t* full = &ring.full[ring.slot];
        const uint32_t bar = moe::smem_addr(full);
        moe::mbar_arrive_expect_tx(full, it.kn > kBox ? 2 * kBoxBytes : kBoxBytes);
        const int group = (int)(weight_row(it, down, a.H, a.I, 0) / 8);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (b * kBox >= it.kn) break;
            const int panel = (it.k0 + b * kBox) * F::kBits / 512;
            if (down)
                box_load_4d(dst + b * kBoxBytes, it.expert < 0 ? &a.m2s : &a.m2, bar, panel, group, policy);
            else
                box_load_5d(dst + b * kBoxBytes, it.expert < 0 ? &a.m13s : &a.m13, bar, panel, group, policy);
        }
    }
    __syncwarp();
    const void* sc = down ? (it.expert < 0 ? a.s2s : a.s2) : (it.expert < 0 ? a.s13s : a.s13);
    if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
        // [gate, up][4 blocks of 128 columns]; phase 2 has one row block
        if (lane < (down ? 4 : 8) && (lane & 3) * 128 < it.kn) {
            const size_t row = weight_row(it, down, a.H, a.I, lane < 4 ? 0 : 8) / 128;
            copy4(dst + 2 * kBoxBytes + lane * 4,
                  static_cast<const float*>(sc) + row * (it.K / 128) + it.k0 / 128 + (lane & 3));
        }
    } else if (DT == MOE_DTYPE_MXFP4_BLOCK32) {
        // 16 bytes a row; they start at a multiple of 16 when K / 32 is one
        const uint8_t* s8 = static_cast<const uint8_t*>(sc);
        if (it.K % 512 == 0 && it.kn == kChunk && it.k0 % 512 == 0) {
#pragma unroll
            for (int r = lane; r < F::kRows; r += 32)
                copy16(dst + 2 * kBoxBytes + r * 16,
                       s8 + (weight_row(it, down, a.H, a.I, r) * it.K + it.k0) / 32);
        } else {
#pragma unroll 4
            for (int i = lane; i < F::kRows * 4; i += 32)
                if ((i & 3) * 128 < it.kn)
                    copy4(dst + 2 * kBoxBytes + i * 4,
                          s8 + (weight_row(it, down, a.H, a.I, i >> 2) * it.K + it.k0) / 32 + (i & 3) * 4);
        }
    }
}

// Producer, all lanes: the activation rows of the stage in `slot`, and the
// lanes' arrival for it.
template <int DT>
__device__ void issue_acts(const FewArgs& a, bool down, uint32_t mask, int base, int count, int k0, int kn,
                           const Ring& ring, int slot) {
    const int lane = threadIdx.x & 31;
    const int xs = x_stride<DT>(chunk_cols(down, count));
    uint32_t dst = moe::smem_addr(ring.base + slot * a.stage_bytes + off_x<DT>());
    if (down) {
        for (int i = 0; i < 2 * count; ++i, dst += xs) {
            const uint16_t* src = (i < count ? a.act_hi + (size_t)(base + i) * a.ld_act
                                             : a.act_lo + (size_t)(base + i - count) * a.ld_act) + k0;
            for (int c = lane * 8; c < kn; c += 256) copy16(dst + c * 2, src + c);
        }
    } else {
        for (uint32_t m = mask; m; m &= m - 1, dst += xs) {
            const uint16_t* src = a.x + (size_t)(__ffs(m) - 1) * a.H + k0;
            for (int c = lane * 8; c < kn; c += 256) copy16(dst + c * 2, src + c);
        }
    }
    arrive_copied(&ring.full[slot]);
}

// ------------------------------------------------------------------ multiplication
// Weights become bf16 pairs whose order the activations' words follow: a
// fragment of two registers, a[0] and a[1], pairs with two activation words.
// (sign | magnitude bits) * 2^E, exact
template <int E>
__device__ __forceinline__ uint32_t merge_sign(uint32_t sign, uint32_t mag) {
    const uint32_t v = (sign & 0x80008000u) | mag;
    constexpr uint32_t kFactor = (uint32_t)(E + 127) << 7 | (uint32_t)(E + 127) << 23;
    const uint32_t f = kFactor;
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&f));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// four e4m3 codes: pairs (0, 2) and (1, 3)
__device__ __forceinline__ void widen_e4m3(uint32_t c, uint32_t& p0, uint32_t& p1, uint32_t& top) {
    const uint32_t m0 = (c << 4) & 0x07f007f0u, m1 = (c >> 4) & 0x07f007f0u;
    p0 = merge_sign<120>(c << 8, m0);
    p1 = merge_sign<120>(c, m1);
    top = __vmaxu2(top, __vmaxu2(m0, m1));   // 0x7f0 is e4m3's NaN
}
// eight e2m1 codes: pairs (0, 4), (1, 5), (2, 6), (3, 7)
__device__ __forceinline__ void widen_e2m1(uint32_t v, uint32_t (&p)[4]) {
    p[0] = merge_sign<126>(v << 12, (v << 6) & 0x01c001c0u);
    p[1] = merge_sign<126>(v << 8, (v << 2) & 0x01c001c0u);
    p[2] = merge_sign<126>(v << 4, (v >> 2) & 0x01c001c0u);
    p[3] = merge_sign<126>(v, (v >> 6) & 0x01c001c0u);
}

// The lane's activations of its column for the warp's 64 columns of K, in
// the weights' order.
template <int DT>
__device__ __forceinline__ void load_acts(const uint8_t* row, int t, uint32_t (&b)[8]) {
    uint4 v[2];
    if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
        // lane t: columns 16 t .. 16 t + 15
        v[0] = *reinterpret_cast<const uint4*>(row + t * 32);
        v[1] = *reinterpret_cast<const uint4*>(row + t * 32 + 16);
    } else {
        // lane t: columns 8 t .. 8 t + 7 of each 32
        v[0] = *reinterpret_cast<const uint4*>(row + t * 16);
        v[1] = *reinterpret_cast<const uint4*>(row + 64 + t * 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 w = v[i];
        uint32_t* o = b + 4 * i;
        if (DT == MOE_DTYPE_BF16) {
            o[0] = w.x;
            o[1] = w.y;
            o[2] = w.z;
            o[3] = w.w;
        } else if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
            o[0] = __byte_perm(w.x, w.y, 0x5410);
            o[1] = __byte_perm(w.x, w.y, 0x7632);
            o[2] = __byte_perm(w.z, w.w, 0x5410);
            o[3] = __byte_perm(w.z, w.w, 0x7632);
        } else {
            o[0] = __byte_perm(w.x, w.z, 0x5410);
            o[1] = __byte_perm(w.x, w.z, 0x7632);
            o[2] = __byte_perm(w.y, w.w, 0x5410);
            o[3] = __byte_perm(w.y, w.w, 0x7632);
        }
    }
}

// One warp's part of a stage: all rows of the unit by its 64 columns of K, for
// NT tiles of 8 tokens.  xrow: the stage's activation row of this lane's
// column, or -1.  In phase 2 a column is a token, and only the expert's own
// tokens add the stage's products: an infinity or a NaN among its weights
// reaches no other.
template <int DT, int NT, bool DOWN>
__device__ __forceinline__ void mma_stage(const Item& it, const uint8_t* stage, int kw, const int (&xrow)[NT],
                                          bool tile1, float (&acc)[Fmt<DT>::kRows / 16][NT][4]) {
    using F = Fmt<DT>;
    constexpr int MT = F::kRows / 16;
    constexpr int PB = kBox * F::kBits / 512;        // 64-byte pieces of a row in a box
    if (kw * kSlice >= it.kn) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int xs = x_stride<DT>(chunk_cols(DOWN, it.count));
    const uint8_t* x = stage + off_x<DT>() + kw * kSlice * 2;
    uint32_t b[NT][8], bl[NT][8];
    bool own[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        own[nt][0] = !DOWN || (it.mask >> (8 * nt + 2 * t) & 1u);
        own[nt][1] = !DOWN || (it.mask >> (8 * nt + 2 * t + 1) & 1u);
        if (nt == 1 && !tile1) continue;
        const uint8_t* xr = x + max(xrow[nt], 0) * xs;
        load_acts<DT>(xr, t, b[nt]);
        if (DOWN) load_acts<DT>(xr + it.count * xs, t, bl[nt]);
    }
    // this warp's columns in the boxes: first piece of 64 bytes
    const int c0 = kw * kSlice;
    const uint8_t* w = stage + (c0 / kBox) * kBoxBytes + (c0 % kBox) * F::kBits / 512 * 512 + g * 64;
    const int sw = (g >> 1) & 3;                     // 64-byte swizzle of row g
    const uint8_t* sc = stage + 2 * kBoxBytes;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const uint8_t* w0 = w + (2 * mt) * PB * 512;
        const uint8_t* w1 = w0 + PB * 512;
        if (DT == MOE_DTYPE_BF16) {
            float c[NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 p = *reinterpret_cast<const uint4*>(w0 + h * 512 + ((t ^ sw) << 4));
                const uint4 q = *reinterpret_cast<const uint4*>(w1 + h * 512 + ((t ^ sw) << 4));
                const uint32_t m0[4] = {p.x, q.x, p.y, q.y}, m1[4] = {p.z, q.z, p.w, q.w};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (nt == 1 && !tile1) continue;
                    mma_bf16(c[nt], m0, b[nt][4 * h], b[nt][4 * h + 1]);
                    mma_bf16(c[nt], m1, b[nt][4 * h + 2], b[nt][4 * h + 3]);
                    if (DOWN) {
                        mma_bf16(c[nt], m0, bl[nt][4 * h], bl[nt][4 * h + 1]);
                        mma_bf16(c[nt], m1, bl[nt][4 * h + 2], bl[nt][4 * h + 3]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (own[nt][j & 1]) acc[mt][nt][j] += c[nt][j];
        } else if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
            const uint4 p = *reinterpret_cast<const uint4*>(w0 + ((t ^ sw) << 4));
            const uint4 q = *reinterpret_cast<const uint4*>(w1 + ((t ^ sw) << 4));
            const uint32_t pc[4] = {p.x, p.y, p.z, p.w}, qc[4] = {q.x, q.y, q.z, q.w};
            const float* fs = reinterpret_cast<const float*>(sc) + c0 / 128;
            const float s0 = fs[0], s1 = DOWN ? s0 : fs[4];
            uint32_t top0 = 0, top1 = 0;
            float c[NT][4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t m[4];
                widen_e4m3(pc[i], m[0], m[2], top0);
                widen_e4m3(qc[i], m[1], m[3], top1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (nt == 1 && !tile1) continue;
                    mma_bf16(c[nt], m, b[nt][2 * i], b[nt][2 * i + 1]);
                    if (DOWN) mma_bf16(c[nt], m, bl[nt][2 * i], bl[nt][2 * i + 1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (own[nt][j & 1]) acc[mt][nt][j] = fmaf(c[nt][j], j < 2 ? s0 : s1, acc[mt][nt][j]);
            // a NaN code anywhere in a row makes its sums NaN
            const uint32_t n0 = __vcmpeq2(top0, 0x07f007f0u), n1 = __vcmpeq2(top1, 0x07f007f0u);
            if (__any_sync(0xffffffffu, n0 | n1)) {
                const bool r0 = __ballot_sync(0xffffffffu, n0 != 0) >> (lane & 28) & 15u;
                const bool r1 = __ballot_sync(0xffffffffu, n1 != 0) >> (lane & 28) & 15u;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (own[nt][j & 1] && (j < 2 ? r0 : r1)) acc[mt][nt][j] = __int_as_float(0x7fc00000);
            }
        } else {
            const uint8_t* sr = sc + (mt * 16 + g) * 16 + kw * 2;
            const uint32_t e0 = *reinterpret_cast<const uint16_t*>(sr);
            const uint32_t e1 = *reinterpret_cast<const uint16_t*>(sr + 128);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // 16-byte piece of the 32-column block, a word a lane
                const int off = ((((c0 >> 5) + h & 3) ^ sw) << 4) + t * 4;
                uint32_t p[4], q[4];
                widen_e2m1(*reinterpret_cast<const uint32_t*>(w0 + off), p);
                widen_e2m1(*reinterpret_cast<const uint32_t*>(w1 + off), q);
                const uint32_t m0[4] = {p[0], q[0], p[1], q[1]}, m1[4] = {p[2], q[2], p[3], q[3]};
                const float s0 = e8m0(e0 >> (8 * h) & 255u), s1 = e8m0(e1 >> (8 * h) & 255u);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (nt == 1 && !tile1) continue;
                    float c[4] = {};
                    mma_bf16(c, m0, b[nt][4 * h], b[nt][4 * h + 1]);
                    mma_bf16(c, m1, b[nt][4 * h + 2], b[nt][4 * h + 3]);
                    if (DOWN) {
                        mma_bf16(c, m0, bl[nt][4 * h], bl[nt][4 * h + 1]);
                        mma_bf16(c, m1, bl[nt][4 * h + 2], bl[nt][4 * h + 3]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (own[nt][j & 1]) acc[mt][nt][j] = fmaf(c[j], j < 2 ? s0 : s1, acc[mt][nt][j]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ the kernel
template <int DT, int NT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
    using F = Fmt<DT>;
    constexpr int R = F::kRows, MT = R / 16, NF = R / 2;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], plan_ready;
    __shared__ int n_active_sh, abort_sh, last_sh;
    float4(*red)[MT][NT][32] = reinterpret_cast<float4(*)[MT][NT][32]>(smem + a.off_red);   // [warp]
    volatile int* abort_flag = &abort_sh;
    Plan P{reinterpret_cast<Active*>(smem + a.off_active), reinterpret_cast<float*>(smem + a.off_pairw),
           &n_active_sh};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.n_stages; ++i) {
            moe::mbar_init(&full[i], 33);       // the weights' bytes, and the producer lanes' copies
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

    if (warp >= kWarps && warp < kWarps + kRouters) {
        // ---------------------------------------------------------- router
        const int tid = threadIdx.x - kGroup, rw = warp - kWarps;
        Scratch S;
        S.keys = reinterpret_cast<double*>(smem + a.off_scratch);
        S.sel = reinterpret_cast<int*>(S.keys + (size_t)min(a.T, kRouters) * a.E);
        S.selw = reinterpret_cast<float*>(S.sel + a.T * a.k);
        S.emask = reinterpret_cast<uint32_t*>(S.selw + a.T * a.k);
        S.apos = reinterpret_cast<int*>(S.emask + a.E);
        for (int i = cta * kRouterGroup + tid; i < a.H / R; i += gridDim.x * kRouterGroup) a.joined[i] = 0;
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
            for (int t = rw; t < a.T; t += kRouters) choose(a, t, S.keys + (size_t)rw * a.E, S);
            group_any(2, false);
            build_plan(a, P, S, tid);
            group_any(2, false);
            if (tid == 0) moe::mbar_arrive(&plan_ready);
        }
    } else if (warp == kWarps + kRouters) {
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
                issue_acts<DT>(a, false, it.mask, 0, it.count, it.k0, it.kn, ring, ring.slot);
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
                for (uint32_t m = __ballot_sync(0xffffffffu, lack); m; m &= m - 1) {
                    const int sl = __ffs(m) - 1;
                    issue_acts<DT>(a, true, 0, __shfl_sync(0xffffffffu, l_base, sl),
                               __shfl_sync(0xffffffffu, l_count, sl), __shfl_sync(0xffffffffu, l_k0, sl),
                               __shfl_sync(0xffffffffu, l_kn, sl), ring, sl);
                }
                lack = 0;
            };
            auto poll = [&]() {
                int n = 0;
                if (lane == 0) {
                    n = *reinterpret_cast<volatile int*>(bars + 1);
                }
                n = __shfl_sync(0xffffffffu, n, 0);
                __threadfence();               // heads and tails are read after the count
                return n >= (int)gridDim.x;
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
                    issue_acts<DT>(a, true, 0, it.base, it.count, it.k0, it.kn, ring, ring.slot);
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
        const int tid = threadIdx.x;
        const int g = lane >> 2, t = lane & 3;
        bool ok = true;
        float acc[MT][NT][4];
        auto clear = [&]() {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;
        };
        // one stage; false when the wait was given up
        auto stage_gate_up = [&](const Item& it) {
            int xrow[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) xrow[i] = 8 * i + g < it.count ? 8 * i + g : 0;
            ok = __all_sync(0xffffffffu, moe::wait_bar(&full[ring.slot], ring.phase, abort_flag, a.status));
            if (!ok) return;
            mma_stage<DT, NT, false>(it, ring.base + ring.slot * a.stage_bytes, warp, xrow, it.count > 8, acc);
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
            ok = __all_sync(0xffffffffu, moe::wait_bar(&full[ring.slot], ring.phase, abort_flag, a.status));
            if (!ok) return;
            mma_stage<DT, NT, true>(it, ring.base + ring.slot * a.stage_bytes, warp, xrow, it.mask >> 8, acc);
            __syncwarp();
            if (lane == 0) moe::mbar_arrive(&empty[ring.slot]);
            ring.next();
        };
        // Leaves the warps' sums in red (once the last ones have been read)
        // and waits for all of them; true when any warp has given up.
        auto gather = [&]() {
            group_any(1, false);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    red[warp][m][i][lane] = make_float4(acc[m][i][0], acc[m][i][1], acc[m][i][2], acc[m][i][3]);
            return group_any(1, !ok);
        };
        // Sum over the K slices, in their order: thread tid takes row tile
        // tid / (32 NT), column tile (tid / 32) % NT.
        auto reduced = [&]() {
            const int m = tid / (32 * NT), i = tid / 32 % NT;
            float4 s = red[0][m][i][lane];
#pragma unroll
            for (int q = 1; q < kWarps; ++q) {
                const float4 v = red[q][m][i][lane];
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
                    // head and tail: together 16 significand bits
                    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                    const __nv_bfloat16 lo = __float2bfloat16_rn(v - __bfloat162float(hi));
                    const size_t at = (size_t)pair * a.ld_act + f;
                    a.act_hi[at] = *reinterpret_cast<const uint16_t*>(&hi);
                    a.act_lo[at] = *reinterpret_cast<const uint16_t*>(&lo);
                }
            }
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
    int split = 148 * kRouters / c->E;
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

// Tensor maps of a matrix stored in bytes, rows of `rb` bytes.  The inner
// dimension is a 64-byte piece of a row, then 8 rows, then the pieces along K
// (zero beyond the row's end), so that a box lands as 512-byte groups of 8
// rows in the 64-byte swizzle.
//   down:    {64, 8, rb / 64, rows / 8},            box {64, 8, PB, R / 8}
//   gate/up: {64, 8, rb / 64, 2, row groups},       box {64, 8, PB, 2, R / 16}
// where the fourth dimension steps from a gate row to its up row.
template <int DT>
moe_status_t few_maps(FewArgs& a, const void* w13, const void* w2, const void* w13s, const void* w2s) {
    using F = Fmt<DT>;
    const uint32_t pb = kBox * F::kBits / 512;
    auto gate_up = [&](CUtensorMap* m, const void* p, uint64_t experts, uint64_t n, const char* what) {
        const uint64_t rb = (uint64_t)a.H * F::kBits / 8;
        const uint64_t dims[5] = {64, 8, rb / 64, 2, (experts * 2 - 1) * n / 8};
        const uint64_t strides[4] = {rb, 64, n * rb, 8 * rb};
        const uint32_t box[5] = {64, 8, pb, 2, F::kRows / 16};
        return moe::api_make_map_u8_sw64(m, p, 5, dims, strides, box, what);
    };
    auto down = [&](CUtensorMap* m, const void* p, uint64_t experts, uint64_t n, const char* what) {
        const uint64_t rb = n * F::kBits / 8;
        const uint64_t dims[4] = {64, 8, rb / 64, experts * a.H / 8};
        const uint64_t strides[3] = {rb, 64, 8 * rb};
        const uint32_t box[4] = {64, 8, pb, F::kRows / 8};
        return moe::api_make_map_u8_sw64(m, p, 4, dims, strides, box, what);
    };
    FEW_TRY(gate_up(&a.m13, w13, a.E, a.I, "w13"));
    FEW_TRY(down(&a.m2, w2, a.E, a.I, "w2"));
    if (a.Is) {
        FEW_TRY(gate_up(&a.m13s, w13s, 1, a.Is, "w13s"));
        FEW_TRY(down(&a.m2s, w2s, 1, a.Is, "w2s"));
    }
    return MOE_OK;
}

// Shared memory: plan, router scratch, the consumers' sums, then as many
// stages as fit.
template <int DT, int NT>
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
    off = up(off + (a.T < kRouters ? a.T : kRouters) * a.E * 8 + n * 8 + a.E * 8, 16);
    a.off_red = off;
    off += kWarps * (F::kRows / 16) * NT * 512;
    a.off_ring = up(off, 1024);
    const int full = kChunk * 2 + F::kPad, half = kBox * 2 + F::kPad;
    const int x = NT == 1 ? 2 * a.T * full : (16 * full > 2 * kT * half ? 16 * full : 2 * kT * half);
    a.stage_bytes = up(off_x<DT>() + x, 512);
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
        FEW_TRY((few_smem<DT, NT>(a, optin - (int)fa.sharedSizeBytes, &smem)));
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
moe_status_t launch_tiles(FewArgs& a, const void* w13, const void* w2, const void* w13s, const void* w2s,
                          cudaStream_t s) {
    FEW_TRY(few_maps<DT>(a, w13, w2, w13s, w2s));
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
    FewArgs a;
    memset(&a, 0, sizeof(a));
    a.x = static_cast<const uint16_t*>(x);
    a.w_router = static_cast<const uint16_t*>(w_router);
    a.bias = bias;
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
        case MOE_DTYPE_BF16: return launch_tiles<MOE_DTYPE_BF16>(a, w13, w2, w13s, w2s, s);
        case MOE_DTYPE_FP8_E4M3_BLOCK128: return launch_tiles<MOE_DTYPE_FP8_E4M3_BLOCK128>(a, w13, w2, w13s, w2s, s);
        default: return launch_tiles<MOE_DTYPE_MXFP4_BLOCK32>(a, w13, w2, w13s, w2s, s);
    }
}

}  // extern "C"
