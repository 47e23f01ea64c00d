// few.cu -- the whole MoE FFN layer for a few tokens in one launch
// (moe_forward_few): router, choice, the experts' SwiGLU and the combine.
//
// Steps a1-a9 of the layer (sources in include/moe.h).  With 1..16 tokens the
// weights of the touched experts are all the traffic and every one is used a
// handful of times, so the kernel is a weight stream: one cooperative launch,
// one block per SM, each block walking its share of the weight rows through a
// shared-memory ring while the multiplications keep up behind it.
//
// Roles in a block (20 warps):
//   warps 0-15  consumers, each with 64 columns of every stage: m16n8k16
//               matrix instructions, 16 weight rows by 8 tokens.  The tokens
//               are the short side; with a few of them the 128-row tiles of
//               tcgen05 would be coarse units to share out over 148 SMs (a
//               decode token touches 1728 16-row units but 216 of 128 rows),
//               and 4- and 8-bit weights are widened in registers.  Warps 8-15
//               first make the choice and the plan of touched experts, while
//               warps 0-7 work on the shared expert, which needs neither
//   warp 16     weight producer: tensor copies of the weights (and scales),
//               stage by stage, as far ahead as the ring is deep
//   warps 17-19 activation producers: the rows that the weights meet (one such
//               warp took 3 % longer with 4-bit weights, two as long as three)
//
// Phases:
//   R   half a block per expert's logits; grid barrier 0; then every block repeats
//       the choice (T * E keys) and the plan
//   1   units of nf SwiGLU features of one expert (nf gate rows, nf up rows,
//       all of K): SiLU(g) * u * w leaves as a bf16 head and a bf16 tail in the
//       workspace; grid barrier 1.  Together they have 16 significand bits: off
//       by 2^-17, 2^-8 of the outputs' own last rounding.  A third part would
//       keep binary32's, with half as many rows again in every stage
//   2   the output rows' sum over all (expert, k) as one long K axis, shared
//       out evenly to 128 columns; a row block that two or more blocks share
//       is joined by the last of them, in block order
// The weight producer does not wait for barrier 1; only the activations do.
//
// 8- and 4-bit weights become binary16 by one conversion for two weights
// (exact: both types lie inside it), and the activations meet them in binary16
// too, lifted: a token, or one unit's features of a SwiGLU output (head and
// tail, 22 significand bits), is scaled by the power of two that takes its
// largest value to 2^14, which keeps every bit of a bf16 value down to 2^-28 of
// the largest and is off by 2^-39 of it below.  A token's lift is undone in
// phase 1's epilogue, a unit's in phase 2 together with the weights' block
// scales.  Phase R lifts the tokens once for all (the shared expert's stages,
// which do not wait for it, lift theirs on the way), phase 1's epilogue its
// outputs.
//
// What it takes and what bounds it (H = 5120, I = 1536, 256 experts, top 8 and
// a shared one, cold L2; in brackets the bytes of the weights that the timed
// tokens touch at the rate of a plain copy, 6.53 TB/s):
//   bf16   1 token 88 us (65): HBM, and 10 us until the choice is known, in
//          which only the shared expert's weights can be fetched; a cooperative
//          launch is 6 us by itself.  16 tokens 659 to 722 us for 78 to 87
//          experts (571 to 636), 5.7 TB/s: the consumers' share of a stage; on
//          78 experts the stream took 593 us without the products (bytes under
//          way are no bound: four stages of 148 blocks are 19 MB).  Tiles of 128
//          rows are the better ones there: moe_forward takes 606 us for 79
//          experts, this kernel 662
//   FP8    1 token 63 us (33): 16 us of launch, router, choice and plan, 7 around
//          grid barrier 1, then HBM and the consumers; without the products 55
//   MXFP4  4 tokens, 28 to 31 experts, 117 to 126 us (56 to 61): the stream with
//          its serial parts (the same 23 us) takes 91 without the products.  With
//          them a warp issues 340 instructions for a stage, 64 of them
//          conversions, and the schedulers issue in 49 % of the cycles: a warp
//          waits for barriers and copies (a quarter of its time, and an eighth in
//          the block's barriers), for the results of ld.shared, conversion and
//          MMA that follow one another (a fifth), and for a busy scheduler or
//          pipe (another fifth)
//   H = 512, I = 128, 32 experts, 1 token: 20.5 us: the launch, two grid
//          barriers of 2 us and code that comes from L2 in every launch
// Tried and not kept: half stages that alternate between the teams (bf16 +4 %,
// FP8 +12 %), looking at the next stage's barriers ahead (+2 %), two reduction
// buffers in turn (0), loading activations only in the lanes that have a token
// (+2 %), the shared expert's down projection fetched into L2 during the choice
// (1 token +1.5 us, 16 tokens -3).
#include "moe.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>
#include <type_traits>

namespace moe {
moe_status_t api_check_config(const moe_config_t* c);
moe_status_t api_fail(moe_status_t st, const char* msg);
void api_clear_error();
moe_status_t api_sm_count(int* n);
moe_status_t api_make_map_u8_sw128(CUtensorMap* m, const void* ptr, uint32_t rank, const uint64_t* dims,
                                  const uint64_t* strides, const uint32_t* box, const char* what);
}  // namespace moe

namespace {

constexpr int kT = MOE_FEW_MAX_T;
constexpr int kWarps = 8;                        // of a team: warps 0-7 (A) and 8-15 (B)
constexpr int kFeeders = 3;                      // warps that copy activations
constexpr int kTeam = kWarps * 32, kConsumers = 2 * kTeam;
constexpr int kThreads = kConsumers + 32 + kFeeders * 32;
constexpr int kOwn = 8;                          // experts of a lane that it chooses from in registers
constexpr int kRouterVecs = 4;                   // 16-byte vectors of a router lane at a time
constexpr int kMaxBlocks = 256;                  // blocks the join buffer has room for
constexpr int kStaticSmem = 4096;                // the kernel's own variables (a launch with less left over fails)
constexpr int kHeadStart = 2;                    // stages copied before barrier 0 has been passed
constexpr int kWindow = 2;                       // stages under way while a barrier or the choice is waited for
// named barriers
constexpr int kBarAll = 1, kBarB = 2, kBarRouted = 3, kBarA = 4, kBarLogits = 5, kBarReaders = 6, kBarLift = 7, kBarTops = 8;
constexpr int kChunk = 1024;                     // K columns of a full stage
constexpr int kBox = 256;                        // K columns of one tensor copy
constexpr int kBoxBytes = 8192;                  // its bytes, for every weight type
constexpr int kSlice = 64;                       // K columns of a warp in a stage
constexpr int kMaxStages = 8;
constexpr float kBf16Max = 0x1.fep+127f;
// Phase 2's sums over 8- and 4-bit weights are held times 2^-kDownShift.  A sum
// of codes times lifted outputs is up to 2^30 (2^15 by 448, 16 columns, 4 sums) and
// what undoes the lift up to 2^113, so it would overflow before it meets the
// weights' scale.  At the other end an output is lifted by at most 2^110, and
// what it and the sums lose is below bf16's smallest value, 2^-133.
constexpr int kDownShift = 16;
constexpr int kBarWord = moe::kSchedFirstWord;   // grid barriers (2) and the exit count, in the status block

// Per weight type: rows of a unit, bits of a weight, bytes of a stage's scales
// and of phase 2's factors (which undo the outputs' lifts), and the activation
// rows' padding.  A stage holds 32 KB of weights, as 128-byte pieces of 8 rows
// (1024 bytes, 128-byte swizzle: 64-byte pieces ran at 5 TB/s at most).  A
// lane's part of a piece, and the padding of the activation rows, are chosen so
// that a load's lanes (8 rows by 4) fall on different banks:
//   bf16   the 16-byte parts 2 t and 2 t + 1: 16 columns in a row
//   e4m3   word t of each 16-byte part: 4 columns of each 16
//   MXFP4  word t of each 16-byte part: 8 columns of each 32
template <int DT>
struct Fmt;
template <>
struct Fmt<MOE_DTYPE_BF16> {
    static constexpr int kRows = 16, kBits = 16, kScaleBytes = 0, kInvBytes = 0, kPad = 16;
};
template <>
struct Fmt<MOE_DTYPE_FP8_E4M3_BLOCK128> {
    static constexpr int kRows = 32, kBits = 8, kScaleBytes = 128, kInvBytes = 1024, kPad = 32;  // scales: [2][8] fp32
};
template <>
struct Fmt<MOE_DTYPE_MXFP4_BLOCK32> {
    static constexpr int kRows = 64, kBits = 4, kScaleBytes = 2048, kInvBytes = 512, kPad = 64;  // [64][32] e8m0
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
    double* logits;             // [T][E]
    uint16_t *act_hi, *act_lo;  // [pairs][ld_act] weighted SwiGLU outputs, head and tail
    uint16_t* x16;              // [T][H] lifted tokens
    float* ainv;                // what undoes the outputs' factors: [pairs][ld_act / features of a unit]
    float* join;                // [blocks][2][T][rows] partial sums of shared row blocks
    int* joined;                // [row blocks] blocks that have left theirs
    int T, H, E, k, I, Is, n_group, topk_group, group_topn, norm, stall, ld_act, batch;
    float rsf;
    unsigned long long inv_g;   // 2^64 / blocks, rounded up
    // shared-memory layout (bytes)
    int off_active, off_pairw, off_pairx, off_cuts, off_scratch, off_red, off_ring, stage_bytes, n_stages;
    int rows_full;              // activation rows of a full stage
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
    float* pairx;      // what undoes its token's lift
    int *cut1, *cut2;  // [blocks + 1] shares of the routed units and of phase 2
    int* n_active;
};

// Scratch of the choice; the consumers' reduction buffer is apart.
struct Scratch {
    unsigned long long* keys;   // [batch][E]
    double* scores;    // the same
    int* sel;          // [T, k]
    double* sels;      // [T, k] their scores
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

// Barrier of both teams (kBarAll) or of one (kBarA, kBarB); true when any of
// their threads says `bad`.
__device__ __forceinline__ bool group_any(int id, bool bad) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)bad), "r"(id == kBarAll ? kConsumers : kTeam)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int n) {
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Shared memory by 32-bit address.
__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t p) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
    return v;
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void bar_done(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A wait that has not been met at once: bounded, and every lane of the warp
// leaves it with the same answer.  `drain`: see moe::wait_bar.
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                                           bool drain) {
    const long long t0 = clock64();
    while (true) {
        if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
        bool stop = !drain && *abort_flag;
        if (clock64() - t0 > moe::kWaitLimit) {
            if (!*abort_flag) atomicOr(status, moe::DEV_STATUS_TIMEOUT);
            *abort_flag = 1;
            stop = true;
        }
        if (__any_sync(0xffffffffu, stop)) return false;
    }
}

// Grid barriers and the join: one thread publishes what its block has written
// (the block's barrier in front of it orders that before), one thread looks,
// and the barrier behind it hands on what it sees.
__device__ __forceinline__ void publish(int* p) {
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}
__device__ __forceinline__ int look(const int* p) {
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int publish_and_acquire(int* p) {
    int v;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Tensor copy of one box, with an L2 policy.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                         int c3, int c4, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
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
__device__ __forceinline__ void arrive_copied(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// D = A B + C: bf16 operands for bf16 weights, binary16 for the others.
template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                      const float (&c)[4]) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
              "f"(c[3]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
              "f"(c[3]));
}

// Two e8m0 scale bytes -> binary32 (0 is 2^-127, 255 NaN): both are bf16 values.
__device__ __forceinline__ void e8m0x2(uint32_t v, float& lo, float& hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}" : "=r"(r) : "r"(v));
    lo = __uint_as_float(r << 16);
    hi = __uint_as_float(r & 0xffff0000u);
}

// ------------------------------------------------------------------ router
// Logits of expert e by one team: a warp sums a slice of K for every token,
// the slices are joined in order.  A product of two bf16 values is exact in
// binary32 (beyond its range an infinity); all sums are binary64, so logits
// whose products are the same in another order are equal wherever the products
// span less than 2^24 or so.  Against sums of eight in binary32 that is 0.1 us
// with one token and 5 of 655 with 16; two tokens at a time cost 2 us of 62 more
// (FP8, one token: code).  `part`: [kWarps][kT] of the team.
__device__ void router_phase(const FewArgs& a, int team, int warp, double (*part)[kT]) {
    const int lane = threadIdx.x & 31, tid = threadIdx.x - team * kTeam;
    const int nch = a.H / 8, per = (nch + kWarps - 1) / kWarps;
    const int c1 = min(nch, (warp + 1) * per);
    for (int e = blockIdx.x + team * gridDim.x; e < a.E; e += 2 * gridDim.x) {
        const uint4* wr = reinterpret_cast<const uint4*>(a.w_router + (size_t)e * a.H);
        bool first = true;
        for (int c0 = warp * per + lane; first || c0 - lane < c1; c0 += 32 * kRouterVecs, first = false) {
            uint4 w[kRouterVecs];
#pragma unroll
            for (int i = 0; i < kRouterVecs; ++i)
                w[i] = c0 + 32 * i < c1 ? __ldg(wr + c0 + 32 * i) : make_uint4(0, 0, 0, 0);
            const uint4* xr = reinterpret_cast<const uint4*>(a.x);
#pragma unroll 1
            for (int t = 0; t < a.T; ++t, xr += nch) {
                uint4 x[kRouterVecs];
#pragma unroll
                for (int i = 0; i < kRouterVecs; ++i)
                    x[i] = c0 + 32 * i < c1 ? __ldg(xr + c0 + 32 * i) : make_uint4(0, 0, 0, 0);
                double sum[kRouterVecs];
#pragma unroll
                for (int i = 0; i < kRouterVecs; ++i) {
                    float wf[8], xf[8];
                    unpack8(w[i], wf);
                    unpack8(x[i], xf);
                    double p[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = (double)__fmul_rn(wf[j], xf[j]);
                    sum[i] = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
                }
                double acc = sum[0];
#pragma unroll
                for (int i = 1; i < kRouterVecs; ++i) acc += sum[i];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
                if (lane == 0) part[warp][t] = first ? acc : part[warp][t] + acc;
            }
        }
        group_any(team ? kBarB : kBarA, false);
        if (tid < a.T) {
            double l = 0.0;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) l += part[q][tid];
            a.logits[(size_t)tid * a.E + e] = l;
        }
        group_any(team ? kBarB : kBarA, false);
    }
}

// Keys are compared as integers in the order of their values; a NaN ranks
// below every number, as -infinity (keys are never -0: a score is not
// negative).
__device__ __forceinline__ unsigned long long sortable(double v) {
    if (isnan(v)) v = -INFINITY;
    const long long b = __double_as_longlong(v);
    return (unsigned long long)(b < 0 ? ~b : b | (1ll << 63));
}
__device__ __forceinline__ double from_sortable(unsigned long long k) {
    return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}

// Warp-wide best of (key, index): larger key first, then lower index; an index
// of 0x7fffffff with key 0 is nobody.  Every lane gets the winner.
__device__ __forceinline__ int warp_best(unsigned long long key, int idx) {
    const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
    const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? lo : 0u);
    return (int)__reduce_min_sync(0xffffffffu, hi == mh && lo == ml ? (uint32_t)idx : 0x7fffffffu);
}

// The choice of token t by one warp, from its E keys and scores.
__device__ void choose(const FewArgs& a, int t, const unsigned long long* key, const double* score,
                       const Scratch& S) {
    const int lane = threadIdx.x & 31;
    uint32_t keep = 0xffffffffu;
    const int gsz = a.E / a.n_group;
    if (a.n_group > 1) {
        // lane g: the sum of group g's group_topn largest keys, largest first
        unsigned long long gs = 0;
        int gi = 0x7fffffff;
        if (lane < a.n_group) {
            double sum = 0.0;
            unsigned long long lk = ~0ull;
            int li = -1;
            for (int j = 0; j < a.group_topn; ++j) {
                unsigned long long bk = 0;
                int bi = 0x7fffffff;
                for (int e = lane * gsz; e < (lane + 1) * gsz; ++e) {
                    const unsigned long long v = key[e];
                    if ((v < lk || (v == lk && e > li)) && v > bk) {
                        bk = v;
                        bi = e;
                    }
                }
                sum = j == 0 ? from_sortable(bk) : sum + from_sortable(bk);
                lk = bk;
                li = bi;
            }
            gs = sortable(sum);
            gi = lane;
        }
        keep = 0;
        for (int j = 0; j < a.topk_group; ++j) {
            const int b = warp_best(gs, gi);
            keep |= 1u << b;
            if (lane == b) {
                gs = 0;
                gi = 0x7fffffff;
            }
        }
    }
    // lane l owns experts l, l + 32, ...
    auto open = [&](int e) { return a.n_group == 1 || (keep >> (e / gsz) & 1u); };
    int my_e = 0;
    if (a.E <= 32 * kOwn) {
        // their keys stay in registers (0: taken, or no expert) and every lane
        // looks its own over again in each turn: E = 256, k = 8 takes 2.0 us
        // where rescanning shared memory in the winner's lane took 3.3
        unsigned long long own[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int e = lane + 32 * i;
            own[i] = e < a.E && open(e) ? key[e] : 0;
        }
        for (int j = 0; j < a.k; ++j) {
            unsigned long long bk = own[0];
            int bi = 0;
#pragma unroll
            for (int i = 1; i < kOwn; ++i)
                if (own[i] > bk) {
                    bk = own[i];
                    bi = i;
                }
            const int e = warp_best(bk, bk ? lane + 32 * bi : 0x7fffffff);
            if (lane == j) my_e = e;
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                if (e == lane + 32 * i) own[i] = 0;
        }
    } else {
        // it rescans them when one is taken
        uint32_t taken = 0;
        unsigned long long bk = 0;
        int bi = 0x7fffffff;
        auto scan = [&]() {
            bk = 0;
            bi = 0x7fffffff;
#pragma unroll 4
            for (int i = 0; i < a.E / 32; ++i) {
                const int e = lane + 32 * i;
                const unsigned long long v = key[e];
                if (!(taken >> i & 1u) && open(e) && v > bk) {
                    bk = v;
                    bi = e;
                }
            }
        };
        scan();
        for (int j = 0; j < a.k; ++j) {
            const int e = warp_best(bk, bi);
            if (lane == j) my_e = e;
            if (lane == (e & 31)) {
                taken |= 1u << (e >> 5);
                scan();
            }
            __syncwarp();
        }
    }
    if (lane < a.k) {
        S.sel[t * a.k + lane] = my_e;
        S.sels[t * a.k + lane] = score[my_e];
        atomicOr(&S.emask[my_e], 1u << t);
    }
}

// ------------------------------------------------------------------ shares
// What block c of G works on.  Phase 1: units of the shared expert (known
// before the choice) and of the routed ones, each cut into G contiguous runs.
// Phase 2: the (row block, expert, K) axis in steps of 128 columns, cut evenly
// (barrier 1 has brought the blocks together).
// c * n / G, rounded down: c n is below 2^37, where the product with
// 2^64 / G, rounded up, has the quotient in its upper half.
__device__ __forceinline__ int cut(const FewArgs& a, int c, int n) {
    return (int)__umul64hi((unsigned long long)c * (unsigned)n, a.inv_g);
}

// Cuts of the routed units and of phase 2, by threads tid of n.
template <int DT>
__device__ void make_cuts(const FewArgs& a, const Plan& P, int n_active, int tid, int n) {
    constexpr int R = Fmt<DT>::kRows;
    const int G = gridDim.x, routed = n_active - (a.Is ? 1 : 0);
    const int us = a.Is / (R / 2), ur = routed * (a.I / (R / 2));
    const int tot2 = a.H / R * (a.Is / 128 + routed * (a.I / 128));
    // Blocks with one shared unit more get one routed unit less, where every
    // block has enough of them for the cuts not to run backwards.
    const bool joint = cut(a, 1, us + ur) >= cut(a, 1, us + G - 1);
#pragma unroll 1
    for (int c = tid; c <= G; c += n) {
        P.cut1[c] = joint ? cut(a, c, us + ur) - cut(a, c, us) : cut(a, c, ur);
        P.cut2[c] = cut(a, c, tot2);
    }
}

// Touched experts in ascending order after the shared one, with their tokens
// and pairs, and the blocks' shares.  Team B; `tid` within it.  Its loops stay
// rolled: the code runs once and comes from L2 in every launch, and rolled the
// tiny layer took 18.7 us where it took 20.0 unrolled.
template <int DT>
__device__ void build_plan(const FewArgs& a, const Plan& P, const Scratch& S, int tid) {
    const int lane = tid & 31, first = a.Is ? 1 : 0;
    // lane l takes experts l * E / 32 and on
    const int per = a.E / 32;
    int n = 0, pairs = 0;
#pragma unroll 2
    for (int i = 0; i < per; ++i) {
        const uint32_t m = S.emask[lane * per + i];
        n += m != 0;
        pairs += __popc(m);
    }
    const int n_active = first + __reduce_add_sync(0xffffffffu, n);
    if (tid < 32) {
        const int n0 = n, p0 = pairs;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, n, off), w = __shfl_up_sync(0xffffffffu, pairs, off);
            if (lane >= off) {
                n += v;
                pairs += w;
            }
        }
        if (lane == 0) *P.n_active = n_active;
        int at = first + n - n0, base = (a.Is ? a.T : 0) + pairs - p0;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            const uint32_t m = S.emask[e];
            if (!m) continue;
            P.active[at] = Active{e, m, base, __popc(m)};
            S.apos[e] = at++;
            base += __popc(m);
        }
        if (a.Is && lane == 0) P.active[0] = Active{-1, (1u << a.T) - 1u, 0, a.T};
    } else {
        make_cuts<DT>(a, P, n_active, tid - 32, kTeam - 32);
    }
}

// Routing weights of the pairs (the producers need not wait for them).
template <bool LIFT>
__device__ void pair_weights(const FewArgs& a, const Plan& P, const Scratch& S, int tid, const uint32_t* lift) {
    for (int i = tid; i < a.T * a.k; i += kTeam) {
        const int t = i / a.k;
        double sum = 0.0;
        for (int j = 0; j < a.k; ++j) sum += S.sels[t * a.k + j];
        const double v = a.norm ? S.sels[i] / sum : S.sels[i];
        const float w = (float)(v * (double)a.rsf);
        const Active act = P.active[S.apos[S.sel[i]]];
        const int pair = act.base + __popc(act.mask & ((1u << t) - 1u));
        P.pairw[pair] = w;
        if (LIFT) P.pairx[pair] = __uint_as_float((254u - lift[t]) << 23);
        if (blockIdx.x == 0) {
            if (a.idx) a.idx[i] = S.sel[i];
            if (a.w) a.w[i] = w;
        }
    }
}

// ------------------------------------------------------------------ the ring
// Slots of a stage, in the order every role walks them; 32-bit addresses.
// Barriers of a slot: `w` and `x`, the weights (and scales) and the activations
// have landed; `empty`, every consumer warp is through.
struct Ring {
    uint32_t w, x, empty, base;
    int n, bytes, scales, slot;   // scales: their offset in a stage
    uint32_t phase;
    // Feeders own slots: whoever waits on a slot's barriers has waited on every
    // turn of it and cannot take an old phase for a new one.
    __device__ __forceinline__ int feeder() const { return slot % kFeeders; }
    __device__ __forceinline__ void next() {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ uint32_t stage() const { return base + slot * bytes; }
};

// Columns of a stage: it has room for rows_full activation rows (heads and
// tails of every pair in phase 2) beside all of its weights; more rows take
// half of the columns, above 16 a quarter.
__device__ __forceinline__ int chunk_cols(const FewArgs& a, bool down, int count) {
    const int rows = down ? 2 * count : count;
    return rows <= a.rows_full ? kChunk : rows <= 16 ? kChunk / 2 : kChunk / 4;
}
template <int DT>
__device__ __forceinline__ int x_stride(int cols) {
    return cols * 2 + Fmt<DT>::kPad;
}
// The activations stand behind the stage's boxes: a stage of fewer columns
// has fewer boxes and room for more rows.
__device__ __forceinline__ int off_x(int cols) { return cols / kBox * kBoxBytes; }

// The stages of phase 1's unit with `count` tokens: stage(k0, kn).
template <class Stage>
__device__ __forceinline__ bool walk_unit(const FewArgs& a, int count, Stage stage) {
    const int cols = chunk_cols(a, false, count);
    for (int k0 = 0; k0 < a.H; k0 += cols)
        if (!stage(k0, min(cols, a.H - k0))) return false;
    return true;
}
__device__ __forceinline__ int unit_stages(const FewArgs& a, int count) {
    const int cols = chunk_cols(a, false, count);
    return (a.H + cols - 1) / cols;
}

// The stages of phase 2's steps begin .. end - 1: item(rb, expert) before the
// stages of an expert, stage(k0, kn), and row_end(rb) behind the last stage of
// a row block (or of the share).  Each returns false to give up.
template <class Item, class Stage, class RowEnd>
__device__ __forceinline__ bool walk_down(const FewArgs& a, const Plan& P, int n_active, int begin, int end,
                                          Item item, Stage stage, RowEnd row_end) {
    if (begin >= end) return true;
    const int first = a.Is ? 1 : 0, ws = a.Is / 128, wi = a.I / 128;
    const int wsum = ws + (n_active - first) * wi;
    int rb = begin / wsum, off = begin - rb * wsum, p = 0;
    if (off >= ws) {
        p = first + (off - ws) / wi;
        off = (off - ws) % wi;
    }
    int pos = begin;
    while (true) {
        const Active act = P.active[p];
        const int steps = act.expert < 0 ? ws : wi, most = chunk_cols(a, true, act.count) / 128;
        if (!item(rb, act)) return false;
        while (off < steps && pos < end) {
            const int n = min(most, min(steps - off, end - pos));
            if (!stage(off * 128, n * 128)) return false;
            off += n;
            pos += n;
        }
        off = 0;
        if (++p == n_active || pos == end) {
            if (!row_end(rb)) return false;
            if (pos == end) return true;
            p = 0;
            ++rb;
        }
    }
}

// Row of its matrix that row r of the unit at feature (or output row) `first`
// is: phase 1 alternates 8 gate rows and the 8 up rows of the same features.
__device__ __forceinline__ size_t gate_up_row(const FewArgs& a, int expert, int first, int r) {
    const int n = expert < 0 ? a.Is : a.I;
    return (expert < 0 ? 0 : (size_t)expert * 2 * n) + first + (r >> 4) * 8 + (r & 7) + (r & 8 ? n : 0);
}
__device__ __forceinline__ size_t down_row(const FewArgs& a, int expert, int first, int r) {
    return (expert < 0 ? 0 : (size_t)expert * a.H) + first + r;
}

// Weight producer: what one unit's (or expert's) stages share.
template <int DT>
struct Source {
    using F = Fmt<DT>;
    const CUtensorMap* map;
    const uint8_t *s0, *s1;     // scales of this lane's rows, at column 0
    int group, K;
    bool down;

    __device__ __forceinline__ void unit(const FewArgs& a, bool dn, int expert, int first) {
        const int lane = threadIdx.x & 31;
        down = dn;
        K = dn ? (expert < 0 ? a.Is : a.I) : a.H;
        map = dn ? (expert < 0 ? &a.m2s : &a.m2) : (expert < 0 ? &a.m13s : &a.m13);
        const uint8_t* sc = static_cast<const uint8_t*>(dn ? (expert < 0 ? a.s2s : a.s2)
                                                           : (expert < 0 ? a.s13s : a.s13));
        auto row = [&](int r) { return dn ? down_row(a, expert, first, r) : gate_up_row(a, expert, first, r); };
        group = (int)(row(0) / 8);
        if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
            // lanes 0-7: the blocks of the gate (or output) rows, 8-15: of the up rows
            s0 = sc + (row(lane & 8 ? 8 : 0) / 128 * (K / 128) + (lane & 7)) * 4;
        } else if (DT == MOE_DTYPE_MXFP4_BLOCK32) {
            s0 = sc + row(lane) * (K / 32);
            s1 = sc + row(lane + 32) * (K / 32);
        }
    }

    // Coordinates of the box at column k (see few_maps): 4-bit rows are one
    // dimension in bytes, the others are cut into 128-byte pieces.
    __device__ __forceinline__ int byte_of(int k) const { return F::kBits == 4 ? k / 2 : 0; }
    __device__ __forceinline__ int piece_of(int k) const { return F::kBits == 4 ? 0 : k * F::kBits / 1024; }

    // All lanes: one tensor copy for each 256 columns, and the scales.
    __device__ __forceinline__ void stage(const Ring& ring, int k0, int kn, uint64_t policy) const {
        const int lane = threadIdx.x & 31;
        const uint32_t dst = ring.stage(), bar = ring.w + 8 * ring.slot;
        if (lane == 0) {
            // A narrow stage's activations stood where this stage's boxes land
            // (off_x): ordinary writes, which the barriers alone do not order
            // before the copies' writes.
            moe::fence_async_smem();
            expect_bytes(bar, (kn + kBox - 1) / kBox * kBoxBytes);
            for (int k = 0; k < kn; k += kBox)
                box_load(dst + k / kBox * kBoxBytes, map, bar, byte_of(k0 + k), 0, piece_of(k0 + k), 0, group, policy);
        }
        const uint32_t sdst = dst + ring.scales;
        if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
            if (lane < (down ? 8 : 16) && (lane & 7) * 128 < kn) copy4(sdst + lane * 4, s0 + k0 / 128 * 4);
            arrive_copied(bar);
        } else if (DT == MOE_DTYPE_MXFP4_BLOCK32) {
            // 16 bytes of a row for 512 columns; they start at a multiple of 16
            // when K / 32 and k0 / 32 do
            for (int k = 0; k < kn; k += 512) {
                const uint8_t *p0 = s0 + (k0 + k) / 32, *p1 = s1 + (k0 + k) / 32;
                const uint32_t d0 = sdst + lane * 32 + k / 32, d1 = d0 + 1024;
                if (kn - k >= 512 && ((K | k0) & 511) == 0) {
                    copy16(d0, p0);
                    copy16(d1, p1);
                } else {
                    for (int j = 0; j < min(512, kn - k) / 32; j += 4) {
                        copy4(d0 + j, p0 + j);
                        copy4(d1 + j, p1 + j);
                    }
                }
            }
            arrive_copied(bar);
        }
    }
};

// Activation producer, all lanes of one warp: a row of kn columns.
__device__ __forceinline__ void copy_row(uint32_t dst, const uint16_t* src, int kn) {
#pragma unroll
    for (int j = 0; j < kChunk / 256; ++j) {
        const int c = (threadIdx.x & 31) * 8 + j * 256;
        if (c < kn) copy16(dst + c * 2, src + c);
    }
}

// Exponent field (biased) of the factor that takes a token's largest value to
// 2^14 .. 2^15, from its bits without the sign: an infinity or NaN counts as
// 2^128, and tiny ones are lifted by at most 2^126.
__device__ __forceinline__ uint32_t lift_of(uint32_t top) { return min(268u - (top >> 7), 253u); }
// Largest of the values' bits (bf16, without the sign).
__device__ __forceinline__ uint32_t top_of(const uint4& v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t lifted(uint32_t w, float f) {
    const float lo = __uint_as_float(w << 16) * f, hi = __uint_as_float(w & 0xffff0000u) * f;
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void put_lifted(uint32_t dst, const uint4& v, float f) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(lifted(v.x, f)), "r"(lifted(v.y, f)),
                 "r"(lifted(v.z, f)), "r"(lifted(v.w, f))
                 : "memory");
}

// A row of the shared expert's stage in binary16, lifted on the way by f.
__device__ __forceinline__ void lift_row(uint32_t dst, const uint16_t* src, int kn, float f) {
    const int lane = threadIdx.x & 31;
    uint4 v[kChunk / 256];
#pragma unroll
    for (int j = 0; j < kChunk / 256; ++j) {
        const int c = lane * 8 + j * 256;
        v[j] = c < kn ? __ldg(reinterpret_cast<const uint4*>(src + c)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kChunk / 256; ++j)
        if (lane * 8 + j * 256 < kn) put_lifted(dst + lane * 16 + j * 512, v[j], f);
}

// The tokens' largest values, by the kFeeders warps: part[warp][token].
__device__ void token_tops(const FewArgs& a, int feeder, uint32_t (*part)[kT]) {
    const int lane = threadIdx.x & 31;
    for (int t = 0; t < a.T; ++t) {
        const uint4* x = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H);
        uint32_t top = 0;
#pragma unroll 8
        for (int c = feeder * 32 + lane; c < a.H / 8; c += kFeeders * 32) top = max(top, top_of(__ldg(x + c)));
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) part[feeder][t] = top;
    }
}

// Phase R: the tokens lifted into the workspace, a warp for 256 columns of one.
__device__ void lift_tokens(const FewArgs& a, int id, int n, const uint32_t* lift) {
    const int lane = threadIdx.x & 31, per = (a.H + 255) / 256;
    for (int u = id; u < a.T * per; u += n) {
        const int t = u / per, c = u % per * 256 + lane * 8;
        if (c >= a.H) continue;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H + c));
        const float f = __uint_as_float(lift[t] << 23);
        *reinterpret_cast<uint4*>(a.x16 + (size_t)t * a.H + c) =
            make_uint4(lifted(v.x, f), lifted(v.y, f), lifted(v.z, f), lifted(v.w, f));
    }
}

// n factors of a row, by the warp.
__device__ __forceinline__ void copy_factors(uint32_t dst, const float* src, int n) {
    for (int i = threadIdx.x & 31; i < n; i += 32) copy4(dst + i * 4, src + i);
}

// ------------------------------------------------------------------ multiplication
// four e4m3 codes -> two binary16 pairs
__device__ __forceinline__ void widen_e4m3(uint32_t v, uint32_t& p0, uint32_t& p1) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(p0), "=r"(p1)
        : "r"(v));
}
// eight e2m1 codes -> four binary16 pairs
__device__ __forceinline__ void widen_e2m1(uint32_t v, uint32_t (&p)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(v));
}

// The lane's activations of its column for the warp's 64 columns of K, in the
// order of the weights' columns.
template <int DT>
__device__ __forceinline__ void load_acts(uint32_t row, int t, uint32_t (&b)[8]) {
    if (DT == MOE_DTYPE_FP8_E4M3_BLOCK128) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 v = lds64(row + j * 32 + t * 8);
            b[2 * j] = v.x, b[2 * j + 1] = v.y;
        }
    } else {
        constexpr bool kWide = DT == MOE_DTYPE_BF16;
        const uint4 v0 = lds128(row + t * (kWide ? 32 : 16));
        const uint4 v1 = lds128(row + (kWide ? t * 32 + 16 : 64 + t * 16));
        b[0] = v0.x, b[1] = v0.y, b[2] = v0.z, b[3] = v0.w;
        b[4] = v1.x, b[5] = v1.y, b[6] = v1.z, b[7] = v1.w;
    }
}

// Which activation rows a lane multiplies in phase 1 (its column's token's
// place in the unit's list) or in phase 2 (a column is a token; one that does
// not use the expert multiplies some row, and its products are dropped).
// Tiles are 8 columns.  With at most four tokens (FOLD) phase 2's tile holds
// the heads in columns 0-3 and the tails in 4-7, which are added at the end;
// otherwise heads and tails are two products.
template <int NT>
struct Columns {
    int x[NT];          // the lane's row in a stage
    int tail;           // from a head to its tail
    int inv[NT][2];     // the factors of the lane's two result columns
    bool own[NT][2];    // the lane's two result columns are the expert's tokens
    bool on[NT];        // the tile has any
};

// Sums of a warp.  `acc` is what its unit (or row block) has so far; bf16
// products need no scale and run on in `run`, two chains, from the first stage
// of an expert to its last.
template <int DT, int NT>
struct Sums {
    static constexpr int MT = Fmt<DT>::kRows / 16;
    static constexpr int RUN = DT == MOE_DTYPE_BF16 ? 2 : 0;
    float acc[MT][NT][4];
    float run[NT][RUN + 1][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;
        restart();
    }
    __device__ __forceinline__ void restart() {
        if constexpr (RUN > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < RUN; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) run[i][h][j] = 0.0f;
        }
    }
    // The expert's products join the columns that are its tokens: an infinity
    // or a NaN among its weights reaches no other.
    __device__ __forceinline__ void fold(const Columns<NT>& col, bool all) {
        if constexpr (RUN > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (all || col.own[i][j & 1]) acc[0][i][j] += run[i][0][j] + run[i][1][j];
            restart();
        }
    }
};

// One warp's part of a stage for one tile of tokens: all rows of the unit by
// 64 columns of K.  A stage with tokens in both tiles does this twice: with 16
// tokens 1.4 of them meet an expert on average, and a branch at every product
// cost more.
template <int DT, int NT, bool DOWN, bool FOLD>
__device__ __forceinline__ void mma_tile(uint32_t stage, uint32_t sc, int slice, const Columns<NT>& col, int nt,
                                         Sums<DT, NT>& sum) {
    using F = Fmt<DT>;
    constexpr int MT = F::kRows / 16;
    constexpr int PB = kBox * F::kBits / 1024;       // 128-byte pieces of a row in a box
    constexpr bool TAIL = DOWN && !FOLD;             // a second product for the tails
    constexpr bool kBf16 = DT == MOE_DTYPE_BF16;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t x = stage + col.x[nt] + slice * (kSlice * 2);
    uint32_t b[8], bl[8];
    load_acts<DT>(x, t, b);
    if (TAIL) load_acts<DT>(x + col.tail, t, bl);
    // row g of the slice's piece; its 16-byte parts are swizzled by the row,
    // and the slice's first part is a multiple of a power of two of them
    constexpr int kParts = kSlice * F::kBits / 128;  // 8, 4, 2
    const int in_box = slice & (kBox / kSlice - 1);
    const uint32_t w = stage + slice / (kBox / kSlice) * kBoxBytes + in_box * kParts / 8 * 1024 + g * 128 +
                       (kBf16 ? 0 : t * 4);
    const int sw = (g ^ (in_box * kParts & 7)) << 4;
    if constexpr (kBf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 p = lds128(w + ((2 * t + h) << 4 ^ sw)), q = lds128(w + PB * 1024 + ((2 * t + h) << 4 ^ sw));
            const uint32_t m0[4] = {p.x, q.x, p.y, q.y}, m1[4] = {p.z, q.z, p.w, q.w};
            float(&c)[4] = sum.run[nt][h];
            mma16<true>(c, m0, b[4 * h], b[4 * h + 1], c);
            mma16<true>(c, m1, b[4 * h + 2], b[4 * h + 3], c);
            if (TAIL) {
                mma16<true>(c, m0, bl[4 * h], bl[4 * h + 1], c);
                mma16<true>(c, m1, bl[4 * h + 2], bl[4 * h + 3], c);
            }
        }
    } else {
        constexpr bool kFp8 = DT == MOE_DTYPE_FP8_E4M3_BLOCK128;
        // Chains of sums with one factor: a token's lift is undone in the
        // epilogue; phase 2 has a factor for a unit's features, 16 (an MMA) or
        // 32 (two), and an e2m1 scale is for 32.
        constexpr int CH = !kFp8 ? 2 : DOWN ? 4 : 1;
        float back[CH][2];              // phase 2: undo the lift of the lane's two result columns
        if (DOWN) {
            const uint32_t inv = sc - F::kInvBytes;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (kFp8) {
                    const uint4 v = lds128(inv + col.inv[nt][j] + slice * 16);
                    const uint32_t f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < CH; ++q) back[q][j] = __uint_as_float(f[q]);
                } else {
                    const uint2 v = lds64(inv + col.inv[nt][j] + slice * 8);
                    back[0][j] = __uint_as_float(v.x), back[1][j] = __uint_as_float(v.y);
                }
            }
        }
        float s0 = 0.0f, s1 = 0.0f;
        if (kFp8) {
            s0 = __uint_as_float(lds32(sc + slice / 2 * 4));
            s1 = DOWN ? s0 : __uint_as_float(lds32(sc + slice / 2 * 4 + 32));
        }
        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const uint32_t w0 = w + (2 * mt) * PB * 1024, w1 = w0 + PB * 1024;
            float c[CH][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t m[2][4];
                if (kFp8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        widen_e4m3(lds32(w0 + ((2 * h + i) << 4 ^ sw)), m[i][0], m[i][2]);
                        widen_e4m3(lds32(w1 + ((2 * h + i) << 4 ^ sw)), m[i][1], m[i][3]);
                    }
                } else {
                    uint32_t p[4], q[4];
                    widen_e2m1(lds32(w0 + (h << 4 ^ sw)), p);
                    widen_e2m1(lds32(w1 + (h << 4 ^ sw)), q);
                    m[0][0] = p[0], m[0][1] = q[0], m[0][2] = p[1], m[0][3] = q[1];
                    m[1][0] = p[2], m[1][1] = q[2], m[1][2] = p[3], m[1][3] = q[3];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    constexpr int kLong = 4 / CH;         // MMAs of a chain
                    float(&d)[4] = c[(2 * h + i) / kLong];
                    if ((2 * h + i) % kLong == 0)
                        mma16<false>(d, m[i], b[4 * h + 2 * i], b[4 * h + 2 * i + 1], zero);
                    else
                        mma16<false>(d, m[i], b[4 * h + 2 * i], b[4 * h + 2 * i + 1], d);
                    if (TAIL) mma16<false>(d, m[i], bl[4 * h + 2 * i], bl[4 * h + 2 * i + 1], d);
                }
            }
            float s[2][2] = {{s0, s1}, {s0, s1}};          // [half][rows g, rows g + 8]
            if (!kFp8) {
                const uint32_t sr = sc + (mt * 16 + g) * 32 + slice * 2;
                e8m0x2(lds16(sr), s[0][0], s[1][0]);
                e8m0x2(lds16(sr + 256), s[0][1], s[1][1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // an infinity or a NaN among the weights reaches the expert's own tokens only
                float v = sum.acc[mt][nt][j];
                if constexpr (kFp8 && DOWN) {
                    float u = c[0][j] * back[0][j & 1];
#pragma unroll
                    for (int q = 1; q < CH; ++q) u = fmaf(c[q][j], back[q][j & 1], u);
                    v = fmaf(u, s[0][j >> 1], v);
                } else {
#pragma unroll
                    for (int q = 0; q < CH; ++q)
                        v = fmaf(DOWN ? c[q][j] * back[q][j & 1] : c[q][j], s[q][j >> 1], v);
                }
                if (!DOWN || col.own[nt][j & 1]) sum.acc[mt][nt][j] = v;
            }
        }
    }
}

template <int DT, int NT, bool DOWN, bool FOLD>
__device__ __forceinline__ void mma_stage(uint32_t stage, uint32_t sc, int slice, const Columns<NT>& col,
                                          Sums<DT, NT>& sum) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        if (NT == 1 || col.on[nt]) mma_tile<DT, NT, DOWN, FOLD>(stage, sc, slice, col, nt, sum);
}

// Warps that the reduction buffer has room for, with 512 bytes a tile: 32 KB at most.
__host__ __device__ constexpr int red_warps(int tiles) { return tiles <= 4 ? 2 * kWarps : kWarps; }

// ------------------------------------------------------------------ the kernel
// NT: tiles of 8 tokens.  FOLD: at most four tokens.
template <int DT, int NT, bool FOLD>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
    using F = Fmt<DT>;
    constexpr int R = F::kRows, MT = R / 16, NF = R / 2, kRedWarps = red_warps(MT * NT);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t bar_w[kMaxStages], bar_x[kMaxStages], bar_empty[kMaxStages], plan_ready;
    __shared__ int n_active_sh, abort_sh, last_sh;
    __shared__ double part[2][kWarps][kT];
    __shared__ uint32_t top_sh[MT][NT][8];
    __shared__ uint32_t x_top[kFeeders][kT], lift_sh[kT];   // of the tokens: largest values, factors
    float4(*red)[MT][NT][32] = reinterpret_cast<float4(*)[MT][NT][32]>(smem + a.off_red);   // [warp]
    volatile int* abort_flag = &abort_sh;
    const Plan P{reinterpret_cast<Active*>(smem + a.off_active), reinterpret_cast<float*>(smem + a.off_pairw),
                 reinterpret_cast<float*>(smem + a.off_pairx),
                 reinterpret_cast<int*>(smem + a.off_cuts), reinterpret_cast<int*>(smem + a.off_cuts) + kMaxBlocks + 1,
                 &n_active_sh};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.n_stages; ++i) {
            moe::mbar_init(&bar_w[i], F::kScaleBytes ? 33 : 1);  // the boxes' bytes, the lanes' scale copies
            moe::mbar_init(&bar_x[i], 32);                       // the lanes' copies
            moe::mbar_init(&bar_empty[i], 2 * kWarps);           // consumer warps
        }
        moe::mbar_init(&plan_ready, 1);
        abort_sh = 0;
        moe::fence_barrier_init();
    }
    __syncthreads();
    // the boxes' swizzle follows the address: 1024-byte alignment of the ring
    Ring ring{moe::smem_addr(bar_w), moe::smem_addr(bar_x), moe::smem_addr(bar_empty),
              (moe::smem_addr(smem) + a.off_ring + 1023) & ~1023u, a.n_stages, a.stage_bytes,
              a.stage_bytes - F::kScaleBytes, 0, 0};
    int* bars = a.status + kBarWord;
    const int cta = blockIdx.x, G = gridDim.x;
    const Active shared{-1, (1u << a.T) - 1u, 0, a.T};
    const int first_routed = a.Is ? 1 : 0, upe = a.I / NF;
    const int s0 = cut(a, cta, a.Is / NF), s1 = cut(a, cta + 1, a.Is / NF);
    const int shared_stages = (s1 - s0) * unit_stages(a, a.T);
    // a wait that every lane of the warp takes and leaves together
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
        return bar_wait_slow(bar, parity, abort_flag, a.status, false);
    };
    const uint32_t plan_bar = moe::smem_addr(&plan_ready);

    if (warp == 2 * kWarps) {
        // ---------------------------------------------------------- weight producer
        const uint64_t policy = moe::l2_policy_evict_first();
        uint32_t issued = 0, last_phase = 0;   // slots in use, and their newest phase
        Source<DT> src;
        int nth = 0;
        bool window = true;
        auto stage = [&](int k0, int kn) {
            if (nth++ == kHeadStart) bar_sync(kBarRouted, kTeam + 32);
            if (!wait(ring.empty + 8 * ring.slot, ring.phase ^ 1)) return false;
            if (window) {
                // more copies under way than HBM's latency needs would only
                // queue, and the router's barrier and loads behind them
                const int back = ring.slot - min(kWindow, ring.n - 1);
                if (!wait(ring.w + 8 * (back < 0 ? back + ring.n : back), back < 0 ? ring.phase ^ 1 : ring.phase))
                    return false;
            }
            src.stage(ring, k0, kn, policy);
            issued |= 1u << ring.slot;
            last_phase = (last_phase & ~(1u << ring.slot)) | (ring.phase << ring.slot);
            ring.next();
            return true;
        };
        bool ok = true;
        for (int u = s0; ok && u < s1; ++u) {
            src.unit(a, false, -1, u * NF);
            ok = walk_unit(a, a.T, stage);
        }
        if (ok && nth <= kHeadStart) {   // not met yet
            bar_sync(kBarRouted, kTeam + 32);
            nth = kHeadStart + 1;
        }
        ok = ok && wait(plan_bar, 0);
        window = false;
        if (ok) {
            for (int u = P.cut1[cta]; ok && u < P.cut1[cta + 1]; ++u) {
                const Active& act = P.active[first_routed + u / upe];
                src.unit(a, false, act.expert, (u % upe) * NF);
                ok = walk_unit(a, act.count, stage);
            }
            // Phase 2 does not wait for barrier 1; until the ring is full its
            // copies leave HBM to the others' last ones and to the barrier.
            window = true;
            int left = a.n_stages;
            ok = ok && walk_down(a, P, n_active_sh, P.cut2[cta], P.cut2[cta + 1],
                                 [&](int rb, const Active& act) {
                                     src.unit(a, true, act.expert, rb * R);
                                     return true;
                                 },
                                 [&](int k0, int kn) {
                                     window = left-- > 0;
                                     return stage(k0, kn);
                                 },
                                 [](int) { return true; });
        }
        // No copy may still be in flight when the block leaves: the consumers
        // may have given up, on the activations, after the last copy was issued.
        for (int i = 0; i < a.n_stages; ++i)
            if (issued >> i & 1u) bar_wait_slow(ring.w + 8 * i, last_phase >> i & 1u, abort_flag, a.status, true);
    } else if (warp > 2 * kWarps) {
        // ---------------------------------------------------------- activation producers
        const int feeder = warp - 2 * kWarps - 1;
        constexpr bool kLift = F::kInvBytes > 0;
        int cols = 0, xs = 0, off = 0;     // of the unit's stages
        bool lifting = kLift;      // the shared expert's tokens are lifted here
        auto factors = [&](int row) {     // of a pair's heads and tails in phase 2, one for a unit's features
            return ring.stage() + ring.scales - F::kInvBytes + row * (cols / NF * 4);
        };
        uint32_t mask = 0;
        auto shape = [&](bool down, int count) {
            cols = chunk_cols(a, down, count);
            xs = x_stride<DT>(cols);
            off = off_x(cols);
        };
        auto stage_x = [&](int k0, int kn) {
            if (ring.feeder() == feeder) {
                if (!wait(ring.empty + 8 * ring.slot, ring.phase ^ 1)) return false;
                uint32_t dst = ring.stage() + off;
                for (uint32_t m = mask; m; m &= m - 1, dst += xs) {
                    const size_t tok = __ffs(m) - 1;
                    if (lifting)
                        lift_row(dst, a.x + tok * a.H + k0, kn, __uint_as_float(lift_sh[tok] << 23));
                    else
                        copy_row(dst, (kLift ? a.x16 : a.x) + tok * a.H + k0, kn);
                }
                if (lifting)
                    bar_done(ring.x + 8 * ring.slot);
                else
                    arrive_copied(ring.x + 8 * ring.slot);
            }
            ring.next();
            return true;
        };
        bool ok = true;
        if (kLift) {
            token_tops(a, feeder, x_top);
            bar_sync(kBarTops, kFeeders * 32);
            if (lane < a.T && feeder == 0) {
                uint32_t top = x_top[0][lane];
#pragma unroll
                for (int i = 1; i < kFeeders; ++i) top = max(top, x_top[i][lane]);
                lift_sh[lane] = lift_of(top);
            }
            bar_sync(kBarTops, kFeeders * 32);
            bar_arrive(kBarLift, kFeeders * 32 + kConsumers);
        }
        mask = shared.mask;
        shape(false, a.T);
        for (int u = s0; ok && u < s1; ++u) ok = walk_unit(a, a.T, stage_x);
        ok = ok && wait(plan_bar, 0);
        lifting = false;
        if (ok) {
            for (int u = P.cut1[cta]; ok && u < P.cut1[cta + 1]; ++u) {
                const Active& act = P.active[first_routed + u / upe];
                mask = act.mask;
                shape(false, act.count);
                ok = walk_unit(a, act.count, stage_x);
            }
            // barrier 1: every block's heads and tails are written
            bool late = false;
            if (ok && lane == 0) {
                const long long t0 = clock64();
                while (look(bars + 1) < G) {
                    if (*abort_flag || clock64() - t0 > moe::kWaitLimit) {
                        if (!*abort_flag) atomicOr(a.status, moe::DEV_STATUS_TIMEOUT);
                        *abort_flag = 1;
                        late = true;
                        break;
                    }
                }
            }
            if (lane == 0) acquire(bars + 1);
            ok = ok && !__any_sync(0xffffffffu, late);
            __syncwarp();
            const uint16_t *hi = nullptr, *lo = nullptr;
            const float* inv = nullptr;
            const int ld_inv = a.ld_act / NF;
            int count = 0;
            if (ok)
                walk_down(a, P, n_active_sh, P.cut2[cta], P.cut2[cta + 1],
                          [&](int, const Active& act) {
                              hi = a.act_hi + (size_t)act.base * a.ld_act;
                              lo = a.act_lo + (size_t)act.base * a.ld_act;
                              inv = a.ainv + (size_t)act.base * ld_inv;
                              count = act.count;
                              shape(true, count);
                              return true;
                          },
                          [&](int k0, int kn) {
                              if (ring.feeder() == feeder) {
                                  if (!wait(ring.empty + 8 * ring.slot, ring.phase ^ 1)) return false;
                                  uint32_t dst = ring.stage() + off;
                                  const uint16_t *h = hi + k0, *l = lo + k0;
                                  const uint32_t tail = (uint32_t)(count * xs);
                                  for (int i = 0; i < count; ++i, dst += xs, h += a.ld_act, l += a.ld_act) {
                                      copy_row(dst, h, kn);
                                      copy_row(dst + tail, l, kn);
                                      if (kLift)
                                          copy_factors(factors(i), inv + (size_t)i * ld_inv + k0 / NF, kn / NF);
                                  }
                                  arrive_copied(ring.x + 8 * ring.slot);
                              }
                              ring.next();
                              return true;
                          },
                          [](int) { return true; });
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ---------------------------------------------------------- consumers
        const int tid = threadIdx.x, g = lane >> 2, t = lane & 3;
        const int team = warp / kWarps, kw = warp % kWarps;
        bool ok = true, good = true;
        Scratch S;
        router_phase(a, team, kw, part[team]);
        if (F::kInvBytes) {
            bar_sync(kBarLift, kFeeders * 32 + kConsumers);
            lift_tokens(a, (2 * kWarps - 1 - warp) * G + cta, 2 * kWarps * G, lift_sh);
        }
        if (team == 0) {
            bar_arrive(kBarLogits, kConsumers);
        } else {
            // ------------------------------------------------------ choice and plan
            const int rid = tid - kTeam;
            S.keys = reinterpret_cast<unsigned long long*>(smem + a.off_scratch);
            S.scores = reinterpret_cast<double*>(S.keys + (size_t)a.batch * a.E);
            S.sels = S.scores + (size_t)a.batch * a.E;
            S.sel = reinterpret_cast<int*>(S.sels + a.T * a.k);
            S.emask = reinterpret_cast<uint32_t*>(S.sel + a.T * a.k);
            S.apos = reinterpret_cast<int*>(S.emask + a.E);
            for (int i = cta * kTeam + rid; i < a.H / R; i += G * kTeam) a.joined[i] = 0;
            for (int e = rid; e < a.E; e += kTeam) S.emask[e] = 0;
            float bias[4];           // of this thread's experts
#pragma unroll
            for (int j = 0; j < 4; ++j) bias[j] = __ldg(a.bias + (rid + j * kTeam) % a.E);
            bar_sync(kBarLogits, kConsumers);
            // barrier 0: every block's logits are written
            if (rid == 0) {
                if (!(a.stall && cta == 0)) publish(bars);
                const long long t0 = clock64();
                while (look(bars) < G) {
                    if (clock64() - t0 > moe::kWaitLimit) {
                        atomicOr(a.status, moe::DEV_STATUS_TIMEOUT);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                }
                acquire(bars);
            }
            good = !group_any(kBarB, !ok);
            bar_arrive(kBarRouted, kTeam + 32);
            if (good) {
                // batch * E is at most 4 kTeam; the next batch's logits are
                // fetched while this one's experts are chosen
                double l[4];
                auto fetch = [&](int t0) {
                    const int n = min(a.batch, a.T - t0) * a.E;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (rid + j * kTeam < n) l[j] = __ldcg(a.logits + (size_t)t0 * a.E + rid + j * kTeam);
                };
                fetch(0);
                for (int t0 = 0; t0 < a.T; t0 += a.batch) {
                    const int nt = min(a.batch, a.T - t0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = rid + j * kTeam;
                        if (i >= nt * a.E) continue;
                        // at -708 exp still has a finite value: scores stay positive, so
                        // that a sum of chosen ones can be divided by (a NaN passes)
                        const double s = 1.0 / (1.0 + exp(l[j] < -708.0 ? 708.0 : -l[j]));
                        S.scores[i] = s;
                        S.keys[i] = sortable(s + (double)bias[j]);
                    }
                    group_any(kBarB, false);
                    if (t0 + a.batch < a.T) fetch(t0 + a.batch);
                    if (kw < nt) choose(a, t0 + kw, S.keys + (size_t)kw * a.E, S.scores + (size_t)kw * a.E, S);
                    group_any(kBarB, false);
                }
                build_plan<DT>(a, P, S, rid);
                group_any(kBarB, false);
                if (rid == 0) moe::mbar_arrive(&plan_ready);
            }
            // the shared expert's stages are the first team's
            ring.slot = shared_stages % a.n_stages;
            ring.phase = (uint32_t)(shared_stages / a.n_stages) & 1u;
        }
        Sums<DT, NT> sum;
        Columns<NT> col = {};
        bool both = false;       // warps 8-15 have joined
        int flip = 0;            // a stage of half the columns goes to one half of the warps, then to the other
        auto release = [&]() {
            __syncwarp();
            // before they join, warps 0-7 answer for warps 8-15 too
            if (lane < (both ? 1 : 2)) bar_done(ring.empty + 8 * ring.slot);
            ring.next();
        };
        // one stage of kn columns; false when a wait was given up
        auto step = [&](auto down, int kn) {
            constexpr bool kDown = decltype(down)::value;
            const uint32_t bw = ring.w + 8 * ring.slot, bx = ring.x + 8 * ring.slot;
            if (!__all_sync(0xffffffffu, bar_try(bw, ring.phase) && bar_try(bx, ring.phase))) {
                ok = wait(bw, ring.phase) && wait(bx, ring.phase);
                if (!ok) return false;
            }
            const uint32_t st = ring.stage();
            if (both) {
                int slice = warp;
                if (kn <= kChunk / 2) {
                    slice = (warp + flip) & 15;
                    flip ^= 8;
                }
                if (slice * kSlice < kn) mma_stage<DT, NT, kDown, FOLD>(st, st + ring.scales, slice, col, sum);
            } else {
                for (int slice = kw; slice * kSlice < kn; slice += kWarps)
                    mma_stage<DT, NT, kDown, FOLD>(st, st + ring.scales, slice, col, sum);
            }
            release();
            return true;
        };
        // Leaves the warps' sums in red (once the last ones have been read)
        // and waits for all of them; true when any warp has given up.  Where
        // the buffer has no room for all 16, warps 8-15 are added to the others.
        auto gather = [&]() {
            const int bar = both ? kBarAll : kBarA;
            group_any(bar, false);
            auto put = [&](int w) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        red[w][m][i][lane] = make_float4(sum.acc[m][i][0], sum.acc[m][i][1], sum.acc[m][i][2],
                                                         sum.acc[m][i][3]);
            };
            if (kRedWarps == 2 * kWarps) {
                put(warp);
            } else {
                if (both) {
                    if (team) put(kw);
                    group_any(bar, false);
                }
                if (!team) {
                    if (both) {
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                const float4 v = red[kw][m][i][lane];
                                sum.acc[m][i][0] += v.x;
                                sum.acc[m][i][1] += v.y;
                                sum.acc[m][i][2] += v.z;
                                sum.acc[m][i][3] += v.w;
                            }
                    }
                    put(kw);
                }
            }
            return group_any(bar, !ok);
        };
        // The sums are joined over the K slices, in their order, by MT * NT
        // warps, one for each row tile and column tile; they take turns.
        int shift = 0;
        auto reader = [&]() {          // 0 .. MT * NT - 1 for the warps whose turn it is
            const int n = both ? 2 * kWarps : kWarps, r = (warp + n - shift) % n;
            shift = (shift + MT * NT) % n;
            return r;
        };
        auto reduced = [&](int r) {
            const int m = r / NT, i = r % NT, n = kRedWarps == 2 * kWarps && both ? 2 * kWarps : kWarps;
            float4 s = red[0][m][i][lane];
#pragma unroll 7
            for (int q = 1; q < n; ++q) {
                const float4 v = red[q][m][i][lane];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            return s;
        };
        auto gate_up = [&](const Active& act, int f0) {
            sum.clear();
            const int count = act.count, cols = chunk_cols(a, false, count);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                col.x[i] = off_x(cols) + (8 * i + g < count ? 8 * i + g : 0) * x_stride<DT>(cols);
                col.on[i] = count > 8 * i;
            }
            walk_unit(a, count, [&](int, int kn) { return step(std::false_type{}, kn); });
            sum.fold(col, true);
            if (gather()) return false;
            if (const int r = reader(); r < MT * NT) {
                const float4 s = reduced(r);
                const int m = r / NT, tile = r % NT, f = f0 + m * 8 + g;
                float gate[2] = {s.x, s.y}, up[2] = {s.z, s.w};
                float v[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = 8 * tile + 2 * t + j;
                    if (F::kInvBytes) {
                        const float back = act.expert < 0 ? __uint_as_float((254u - lift_sh[c < count ? c : 0]) << 23)
                                                          : P.pairx[act.base + (c < count ? c : 0)];
                        gate[j] *= back, up[j] *= back;
                    }
                    v[j] = gate[j] / (1.0f + expf(-gate[j])) * up[j];
                    if (act.expert >= 0) v[j] *= P.pairw[act.base + (c < count ? c : 0)];
                }
                if constexpr (F::kInvBytes > 0) {
                    // one factor for the unit's features: the readers of its
                    // row tiles exchange their largest
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t top = __float_as_uint(v[j]) & 0x7fffffffu;
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                        if (g == 0) top_sh[m][tile][2 * t + j] = top;
                    }
                    bar_sync(kBarReaders, MT * NT * 32);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = 8 * tile + 2 * t + j;
                        if (c >= count) continue;
                        uint32_t top = top_sh[0][tile][2 * t + j];
#pragma unroll
                        for (int q = 1; q < MT; ++q) top = max(top, top_sh[q][tile][2 * t + j]);
                        const uint32_t lift = min(268u - (top >> 23), 253u - kDownShift);
                        // head and tail: together 22 significand bits; an infinity has no tail
                        const float x = v[j] * __uint_as_float(lift << 23);
                        const __half hi = __float2half_rn(x);
                        const __half lo = __float2half_rn(isinf(x) ? 0.0f : x - __half2float(hi));
                        const size_t pair = act.base + c, at = pair * a.ld_act + f;
                        a.act_hi[at] = __half_as_ushort(hi);
                        a.act_lo[at] = __half_as_ushort(lo);
                        if (m == 0 && g == 0)
                            a.ainv[pair * (a.ld_act / NF) + f0 / NF] = __uint_as_float((254u - kDownShift - lift) << 23);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = 8 * tile + 2 * t + j;
                        if (c >= count) continue;
                        // head and tail: together 16 significand bits.  Above bf16's largest
                        // value the tail takes the rest; an infinity has no tail, and a NaN
                        // is in the tail at least.
                        const bool inf = isinf(v[j]);
                        const float top = fminf(fmaxf(v[j], -kBf16Max), kBf16Max);
                        const __nv_bfloat16 hi = __float2bfloat16_rn(inf ? v[j] : top);
                        const __nv_bfloat16 lo = __float2bfloat16_rn(inf ? 0.0f : v[j] - __bfloat162float(hi));
                        const size_t at = (size_t)(act.base + c) * a.ld_act + f;
                        a.act_hi[at] = __bfloat16_as_ushort(hi);
                        a.act_lo[at] = __bfloat16_as_ushort(lo);
                    }
                }
            }
            return true;
        };

        if (team == 0)
            for (int u = s0; good && u < s1; ++u) good = gate_up(shared, u * NF);
        if (good) ok = wait(plan_bar, 0);
        good = !group_any(kBarAll, !(good && ok));
        both = true;
        shift = 0;
        if (good && team) pair_weights<(F::kInvBytes > 0)>(a, P, S, tid - kTeam, lift_sh);   // read behind gather's barriers
        if (good)
            for (int u = P.cut1[cta]; good && u < P.cut1[cta + 1]; ++u)
                good = gate_up(P.active[first_routed + u / upe], (u % upe) * NF);
        if (good) {
            // barrier 1: this block's heads and tails are written
            group_any(kBarAll, false);
            if (tid == 0) publish(bars + 1);
            const int begin = P.cut2[cta], end = P.cut2[cta + 1];
            const int wsum = a.Is / 128 + (n_active_sh - first_routed) * (a.I / 128);
            sum.clear();
            auto item = [&](int, const Active& act) {
                sum.fold(col, false);   // the last expert's
                const int cols = chunk_cols(a, true, act.count), xs = x_stride<DT>(cols);
                col.tail = act.count * xs;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int tok = FOLD ? g & 3 : 8 * i + g;
                    const bool has = act.mask >> tok & 1u;
                    const int row = __popc(act.mask & ((1u << tok) - 1u)) + (FOLD && g >= 4 ? act.count : 0);
                    col.x[i] = off_x(cols) + (has ? row * xs : 0);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = FOLD ? (2 * t + j) & 3 : 8 * i + 2 * t + j;
                        col.own[i][j] = act.mask >> c & 1u;
                        col.inv[i][j] = col.own[i][j] ? __popc(act.mask & ((1u << c) - 1u)) * (cols / NF * 4) : 0;
                    }
                    col.on[i] = act.mask >> (8 * i) & 255u;
                }
                return true;
            };
            // a given-up wait ends in row_end, which all warps reach
            auto stage = [&](int, int kn) {
                if (ok) step(std::true_type{}, kn);
                return true;
            };
            auto row_end = [&](int rb) {
                sum.fold(col, false);
                if (gather()) return false;
                const int lo = rb * wsum, hi = lo + wsum;
                const bool whole = begin <= lo && hi <= end;
                float* mine = a.join + ((size_t)cta * 2 + (begin >= lo ? 0 : 1)) * a.T * R;
                if (const int rd = reader(); rd < MT * NT) {
                    float4 s = reduced(rd);
                    if (FOLD) {   // columns 4-7 hold the tails' sums of columns 0-3
                        s.x += __shfl_down_sync(0xffffffffu, s.x, 2);
                        s.y += __shfl_down_sync(0xffffffffu, s.y, 2);
                        s.z += __shfl_down_sync(0xffffffffu, s.z, 2);
                        s.w += __shfl_down_sync(0xffffffffu, s.w, 2);
                    }
                    const int r = rd / NT * 16 + g, c0 = rd % NT * 8 + 2 * t;
                    constexpr float kUp = F::kInvBytes ? (float)(1 << kDownShift) : 1.0f;
                    const float v[4] = {s.x * kUp, s.y * kUp, s.z * kUp, s.w * kUp};
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
                sum.clear();
                if (whole) return true;
                // a row block of several blocks: the last to leave its part
                // adds them up in block order
                int c0 = cta, c1 = cta + 1;
                while (P.cut2[c0] > lo) --c0;
                while (P.cut2[c1] < hi) ++c1;
                int parts = 0;
                for (int c = c0; c < c1; ++c) parts += P.cut2[c] < P.cut2[c + 1];
                group_any(kBarAll, false);
                if (tid == 0) last_sh = publish_and_acquire(a.joined + rb) == parts - 1;
                group_any(kBarAll, false);
                if (last_sh) {
                    for (int i = tid; i < a.T * R; i += kConsumers) {
                        float s = 0.0f;
                        for (int c = c0; c < c1; ++c)
                            if (P.cut2[c] < P.cut2[c + 1])
                                s += __ldcg(a.join + ((size_t)c * 2 + (P.cut2[c] >= lo ? 0 : 1)) * a.T * R + i);
                        const __nv_bfloat16 b = __float2bfloat16_rn(s);
                        a.out[(size_t)(i / R) * a.H + rb * R + i % R] = *reinterpret_cast<const uint16_t*>(&b);
                    }
                }
                return true;   // gather's first barrier keeps last_sh until every thread has read it
            };
            walk_down(a, P, n_active_sh, begin, end, item, stage, row_end);
        }
    }
    __syncthreads();
    // the last block to leave clears the counters for the next launch
    if (threadIdx.x == 0 && atomicAdd(bars + 2, 1) == G - 1) {
        bars[0] = 0;
        bars[1] = 0;
        bars[2] = 0;
    }
}

// ------------------------------------------------------------------ host side
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct FewLayout {
    size_t logits, hi, lo, x16, ainv, join, joined, total;
    int ld_act;
};

FewLayout few_layout(const moe_config_t* c) {
    FewLayout L{};
    const int Is = c->n_shared * c->I;
    L.ld_act = Is > c->I ? Is : c->I;
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = up256(off + bytes);
        return at;
    };
    L.logits = take((size_t)c->T * c->E * 8);
    L.hi = take((size_t)c->T * (c->k + 1) * L.ld_act * 2);
    L.lo = take((size_t)c->T * (c->k + 1) * L.ld_act * 2);
    L.x16 = take((size_t)c->T * c->H * 2);
    L.ainv = take((size_t)c->T * (c->k + 1) * (L.ld_act / 16) * 4);
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
    // the shares are counted in 32 bits: steps of 16 rows by 128 columns
    const long long act = (long long)c->T * c->k + c->n_shared, blocks = (long long)(c->H / 16) * (c->I / 128);
    if (act * blocks > (1ll << 28) || act * (c->I / 8) > (1ll << 22) || (long long)c->E * 2 * c->I > (1ll << 31))
        return ffail(MOE_ERR_UNSUPPORTED, "%s H=%lld, I=%lld too large", "few-token layer:", c->H, c->I);
    return MOE_OK;
}

// What the call writes may overlap nothing else but out x.
moe_status_t few_apart(const moe_config_t* c, const void* x, const void* w_router, const float* bias, const void* w13,
                       const void* s13, const void* w2, const void* s2, const void* w13s, const void* s13s,
                       const void* w2s, const void* s2s, const void* out, const int32_t* idx, const float* w,
                       const void* ws, size_t ws_bytes) {
    const size_t n = (size_t)c->T * c->H * 2, Is = (size_t)c->n_shared * c->I, nk = (size_t)c->T * c->k * 4;
    const size_t routed = (size_t)c->E * c->H * c->I, shared = (size_t)c->H * Is;   // elements of a down projection
    auto stored = [&](size_t v) {
        return c->dtype == MOE_DTYPE_BF16 ? 2 * v : c->dtype == MOE_DTYPE_MXFP4_BLOCK32 ? v / 2 : v;
    };
    auto scales = [&](size_t v) { return c->dtype == MOE_DTYPE_MXFP4_BLOCK32 ? v / 32 : v / (128 * 128) * 4; };
    const moe::Span in[] = {{x, n, "x"},
                            {w_router, (size_t)c->E * c->H * 2, "w_router"},
                            {bias, (size_t)c->E * 4, "bias"},
                            {w13, stored(2 * routed), "w13"},
                            {s13, scales(2 * routed), "w13_scale"},
                            {w2, stored(routed), "w2"},
                            {s2, scales(routed), "w2_scale"},
                            {w13s, stored(2 * shared), "w13s"},
                            {s13s, scales(2 * shared), "w13s_scale"},
                            {w2s, stored(shared), "w2s"},
                            {s2s, scales(shared), "w2s_scale"}};
    const moe::Span outs[] = {{out, n, "out"}, {idx, nk, "topk_idx"}, {w, nk, "topk_w"}, {ws, ws_bytes, "the workspace"}};
    for (const moe::Span& o : outs) {
        for (const moe::Span& i : in)
            if (moe::overlap(o, i) && !(&o == outs && &i == in && o.p == i.p))
                return ffail(MOE_ERR_INVALID_ARG, "%s overlaps a buffer of the call", o.name);
        for (const moe::Span& q : outs)
            if (&q > &o && moe::overlap(o, q)) return ffail(MOE_ERR_INVALID_ARG, "%s overlaps a buffer of the call", o.name);
    }
    return MOE_OK;
}

// Tensor maps of a matrix stored in bytes, rows of `rb` bytes, all of five
// dimensions.  A box of 256 columns lands as 128-byte pieces of 8 rows (1024
// bytes, 128-byte swizzle), the pieces along K inside 8-row groups:
//   {128, 8, rb / 128, halves, row groups}, box {128, 8, PB, halves, groups of a unit}
// `halves` steps from a gate row to its up row (1 for the down matrix).  A
// 4-bit row may end inside a piece, so there the first dimension is the whole
// row and a box one piece of it ({rb, 8, 1, halves, row groups}); beyond a
// row's end a box is filled with zeros.
template <int DT>
moe_status_t few_maps(FewArgs& a, const void* w13, const void* w2, const void* w13s, const void* w2s) {
    using F = Fmt<DT>;
    const bool whole = F::kBits == 4;
    auto map = [&](CUtensorMap* m, const void* p, uint64_t K, uint64_t groups, uint32_t halves, uint64_t n,
                   const char* what) {
        const uint64_t rb = K * F::kBits / 8;
        const uint64_t dims[5] = {whole ? rb : 128, 8, whole ? 1 : rb / 128, halves, groups};
        const uint64_t strides[4] = {rb, 128, n * rb, 8 * rb};
        const uint32_t box[5] = {128, 8, whole ? 1u : (uint32_t)kBox * F::kBits / 1024, halves,
                                 F::kRows / 8 / halves};
        return moe::api_make_map_u8_sw128(m, p, 5, dims, strides, box, what);
    };
    auto gate_up = [&](CUtensorMap* m, const void* p, uint64_t experts, uint64_t n, const char* what) {
        return map(m, p, a.H, (experts * 2 - 1) * n / 8, 2, n, what);
    };
    auto down = [&](CUtensorMap* m, const void* p, uint64_t experts, uint64_t n, const char* what) {
        return map(m, p, n, experts * a.H / 8, 1, 8, what);
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
    off += (n + a.T) * 4;
    a.off_pairx = off;
    if (F::kInvBytes) off += (n + a.T) * 4;
    a.off_cuts = off;
    off = up(off + 2 * (kMaxBlocks + 1) * 4, 16);
    a.off_scratch = off;
    // tokens chosen at a time, so that their keys and scores stay within 16 KB
    const int most = a.E <= 256 ? 4 : a.E <= 512 ? 2 : 1;
    a.batch = a.T < most ? a.T : most;
    off = up(off + a.batch * a.E * 16 + n * 12 + a.E * 8, 16);
    a.off_red = off;
    constexpr int tiles = F::kRows / 16 * NT;
    off += red_warps(tiles) * tiles * 512;
    a.off_ring = up(off, 1024);
    // As many stages as there is room for with four activation rows in a full
    // one (most experts have one or two tokens), then as many rows, up to
    // eight, as these stages have room for.  (16 tokens, bf16: three stages of
    // eight rows took 690 us, four of four 663; where the tokens crowd onto few
    // experts, more rows than a full stage holds cost half stages: 8 tokens
    // 502 us with four rows, 412 with seven.  Up to four tokens only the shared
    // expert has more than two, and MXFP4 took 123 us with eight rows, 119 with
    // four.)
    auto bytes_of = [&](int rows) {
        return up(kChunk / kBox * kBoxBytes + rows * (kChunk * 2 + F::kPad) + F::kInvBytes + F::kScaleBytes, 1024);
    };
    const int room = limit - 1024 - a.off_ring;   // 1024: the boxes' alignment
    a.rows_full = a.T == 1 ? 2 : 4;
    const int all = a.T <= 4 ? a.rows_full : 8;
    const int stages = room / bytes_of(a.rows_full);
    a.n_stages = stages < kMaxStages ? stages : kMaxStages;
    while (a.rows_full < all && a.n_stages * bytes_of(a.rows_full + 1) <= room) ++a.rows_full;
    a.stage_bytes = bytes_of(a.rows_full);
    if (a.n_stages < 2)
        return ffail(MOE_ERR_UNSUPPORTED, "%s: %lld bytes of shared memory hold too few stages", "few-token layer",
                     limit);
    *bytes = 1024 + (size_t)a.off_ring + (size_t)a.n_stages * a.stage_bytes;
    return MOE_OK;
}

template <int DT, int NT, bool FOLD>
moe_status_t launch_few(FewArgs& a, cudaStream_t s) {
    void (*kernel)(FewArgs) = few_kernel<DT, NT, FOLD>;
    int sms = 0, dev = 0, optin = 0;
    FEW_TRY(moe::api_sm_count(&sms));
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) {
        size_t smem = 0;
        FEW_TRY((few_smem<DT, NT>(a, optin - kStaticSmem, &smem)));
        // the kernel's limit is the process's: always the same one, or a call of
        // another size in another thread could lower it before this launch
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - kStaticSmem);
        if (e == cudaSuccess) {
            void* args[] = {&a};
            const int grid = sms < kMaxBlocks ? sms : kMaxBlocks;
            a.inv_g = ~0ull / grid + 1;
            e = cudaLaunchCooperativeKernel(kernel, dim3(grid), dim3(kThreads), args, smem, s);
        }
    }
    if (e != cudaSuccess) return ffail(MOE_ERR_CUDA, "few-token layer launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

template <int DT>
moe_status_t launch_tiles(FewArgs& a, const void* w13, const void* w2, const void* w13s, const void* w2s,
                          cudaStream_t s) {
    FEW_TRY(few_maps<DT>(a, w13, w2, w13s, w2s));
    if (a.T <= 4) return launch_few<DT, 1, true>(a, s);
    return a.T <= 8 ? launch_few<DT, 1, false>(a, s) : launch_few<DT, 2, false>(a, s);
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
    // out may be x: it is written when every block has read its tokens
    FEW_TRY(few_apart(cfg, x, w_router, bias, w13, w13_scale, w2, w2_scale, shared ? w13s : nullptr, w13s_scale,
                      shared ? w2s : nullptr, w2s_scale, out, topk_idx, topk_w, ws, L.total));
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
    a.logits = reinterpret_cast<double*>(base + L.logits);
    a.act_hi = reinterpret_cast<uint16_t*>(base + L.hi);
    a.act_lo = reinterpret_cast<uint16_t*>(base + L.lo);
    a.x16 = reinterpret_cast<uint16_t*>(base + L.x16);
    a.ainv = reinterpret_cast<float*>(base + L.ainv);
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
