// kda_fp8_matmul.cu -- products of e4m3 rows and e4m3 weights with an fp32 scale for every 128 elements along K.
//
//   out[m, n] = sum_b xs[m, b] ws[n, b] sum_{k in block b} x[m, k] w[n, k]
//
// A tile of 128 x TN outputs: rows p of the first operand (a matrix instruction's M) by rows q of the second (its N).  With many
// rows of x, p is a row of x and q one of w; with few, the other way about (SWAP), so that the 128 rows of an instruction are
// filled by the weights, whose bytes are all that counts then.  tcgen05 forms one block's 128 x TN x 128 product at a time in
// TMEM (two accumulators by turns); the epilogue's warps take it from there into fp32 registers, times the block's scales, while the
// next block is multiplied.  The scales cannot go into the operands without a second rounding, and the sum over blocks in
// registers is an fma in fp32.  8192 x 8192 x 4096: 230 us, 2.4 PFLOP/s, the tensor pipe 55 % busy: bound by the accumulators' way from
// products to registers and back.  16 x 8192 x 4096: 12 us, of which the weights' bytes are 5.
#include <cuda_bf16.h>

#include <algorithm>

#include "kda_fp8_internal.h"
#include "kda_gdn_ptx.cuh"

namespace kda {
namespace {

constexpr int kTileP = 128;
constexpr int kMaxSplit = 8;

// D[tmem] (+)= A[smem desc] B[smem desc], e4m3 operands (32 of K), fp32 accumulate.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// ------------------------------------------------------------ pairs of blocks --
// Two blocks of a cluster multiply together (cta_group::2): 256 rows of P, 128 from each, by TN of Q, half of them in each one's
// shared memory, so a block loads half as much of Q.  The first one issues; barriers in it are the pair's.
__device__ __forceinline__ void pair_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` of both blocks when every product issued so far by this thread is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* slot, uint32_t ncols) {  // whole warp, in both
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {  // whole warp, in both
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// A load into this block's shared memory, counted on a barrier of the pair's (an address in the cluster).
__device__ __forceinline__ void pair_tma_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// What it orders is reads of TMEM, which tcgen05's fences order; a release of the cluster would wait for all of the warp's stores.
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Instruction descriptor, kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (bits 7-9 and 10-12 = 0), both K-major (bits 15, 16),
// N >> 3 in bits 17-22, M >> 4 in bits 24-28.
constexpr uint32_t idesc_e4m3(int M, int N) { return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24); }

// The wait for tcgen05.ld, tied to the registers that it fills.
__device__ __forceinline__ void tmem_ld_wait16(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                   "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])::"memory");
}

// Two floats as the register pair that f32x2 instructions take.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void fma2(float* sum, const float* v, uint64_t scale) {  // sum += v scale
    uint64_t s = pair_of(sum[0], sum[1]);
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(pair_of(v[0], v[1])), "l"(scale));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(sum[0]), "=f"(sum[1]) : "l"(s));
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

__device__ __forceinline__ void cluster_store(uint32_t addr, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

constexpr int kQuad = 4;  // blocks of K whose scales are copied together: 16 bytes of a row's, one sector of L2 for all

template <int TN, bool PAIR>
struct Shape {
    static constexpr int kQ = TN / (PAIR ? 2 : 1);                // rows of Q in a block's shared memory
    static constexpr int kWarps = TN >= 64 ? TN / 16 : 4;         // of the epilogue: a quarter of the rows each

    static constexpr int kCols = TN / (kWarps / 4);               // of an epilogue thread
    static constexpr int kStage = (kTileP + kQ) * kFp8Block;      // bytes of a K block's operands
    // As many as leave room for kBlocks; a fifth of the pairs' cost 1 % (8192 x 8192 x 4096, scales by rows: 384 us against 368).
    static constexpr int kStages = TN == 64 || PAIR ? 4 : 5;
    static constexpr int kCopy = kWarps, kScales = kWarps + 1, kMultiply = kWarps + 2;  // the other warps
    static constexpr int kThreads = 32 * (kMultiply + 1);
    static constexpr int kScaleStages = (kStages + 2) / kQuad + 2;  // quads of blocks: copies run this far ahead of the epilogue
    static constexpr int kTmem = 2 * TN < 32 ? 32 : 2 * TN;
    static constexpr int kBlocks = TN >= 128 ? 1 : 2;             // on an SM
    static constexpr int kStaged = 64;                            // bytes of a row that a warp turns over at once on its way out
};
template <int TN, bool PAIR>
struct Shared {
    using S = Shape<TN, PAIR>;
    uint64_t full[S::kStages], empty[S::kStages];
    uint64_t scale_full[S::kScaleStages], scale_empty[S::kScaleStages];
    uint64_t done[2], taken[2];  // accumulators: multiplied, read
    uint64_t drained;
    uint32_t tmem;
    int32_t stop;
    alignas(16) float p_scale[S::kScaleStages][kTileP][kQuad];
    alignas(16) float q_scale[S::kScaleStages][kQuad][TN];
    alignas(16) uint8_t staged[PAIR ? S::kWarps : 1][PAIR ? 32 * S::kStaged : 16];
};
template <int TN, bool PAIR>
constexpr uint32_t smem_bytes() {
    return Shape<TN, PAIR>::kStages * Shape<TN, PAIR>::kStage + 1024 + static_cast<uint32_t>(sizeof(Shared<TN, PAIR>));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// A wait that gives up after kWaitLimit or once another one of the block has.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int32_t* stop, int32_t* status) {
    if (kWaitLimit == 0 ? mbar_test(bar, parity) : mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (kWaitLimit != 0 && !*stop && clock64() - t0 <= kWaitLimit)
        if (mbar_try_wait(bar, parity)) return true;
    if (!*stop && status) atomicOr(status, KDA_DEV_TIMEOUT);
    *stop = 1;
    return false;
}
// The same by a whole warp, with one answer.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int32_t* stop, int32_t* status) {
    return __all_sync(~0u, wait_one(bar, parity, stop, status));
}

// The tiles of all experts, one after the other; whole warp.
struct Tile {
    int32_t expert, p0, q0;  // first row of w's expert or of x, by the operand that it is of
    int32_t row_end;         // behind the expert's rows of x
    int32_t blocks;          // of K
};
template <int TN, bool PAIR>
struct Walk {
    static constexpr bool SWAP = !PAIR;
    int32_t e0 = 0;       // the experts looked at start here
    int64_t before = 0;   // tiles of those before
    __device__ __forceinline__ bool find(const Fp8MatmulArgs& a, int32_t tile, Tile* t) {
        const int lane = threadIdx.x & 31;
        const int32_t along_w = (a.N + (SWAP ? kTileP : TN) - 1) / (SWAP ? kTileP : TN);
        constexpr int kP = kTileP * (PAIR ? 2 : 1), kRows = SWAP ? TN : kP;
        int32_t lo = 0, hi = a.rows;
        if (a.offsets) {
            if (tile >= (a.rows / kRows + a.experts) * along_w) return false;  // more than rows in order have, and int32 holds
            for (;;) {
                if (e0 >= a.experts) return false;
                const int32_t e = e0 + lane;
                lo = hi = 0;
                if (e < a.experts) {  // offsets that fall or leave the rows give fewer rows, none outside
                    lo = min(max(__ldg(a.offsets + e), 0), a.rows);
                    hi = max(lo, min(__ldg(a.offsets + e + 1), a.rows));
                }
                const int64_t own = static_cast<int64_t>((hi - lo + kRows - 1) / kRows) * along_w;
                int64_t sum = own;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int64_t up = __shfl_up_sync(~0u, sum, d);
                    if (lane >= d) sum += up;
                }
                const uint32_t past = __ballot_sync(~0u, before + sum > tile);
                if (past) {
                    const int at = __ffs(past) - 1;
                    tile -= static_cast<int32_t>(before + __shfl_sync(~0u, sum - own, at));
                    lo = __shfl_sync(~0u, lo, at);
                    hi = __shfl_sync(~0u, hi, at);
                    t->expert = e0 + at;
                    break;
                }
                before += __shfl_sync(~0u, sum, 31);
                e0 += 32;
            }
        } else {
            if (tile >= static_cast<int64_t>((a.rows + kRows - 1) / kRows) * along_w) return false;
            t->expert = 0;
        }
        const int32_t along_p = SWAP ? along_w : (hi - lo + kP - 1) / kP;
        const int32_t q = static_cast<int32_t>(static_cast<uint32_t>(tile) / static_cast<uint32_t>(along_p)), p = tile - q * along_p;
        t->p0 = SWAP ? p * kP : lo + p * kP;
        t->q0 = SWAP ? lo + q * TN : q * TN;
        t->row_end = hi;
        return true;
    }
};

__device__ __forceinline__ void store1(const Fp8MatmulArgs& a, int64_t at, float v) {
    if (a.out_f32) static_cast<float*>(a.out)[at] = v;
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

// PER_Q: a scale for every q, else one for 128 of them.  gridDim = clusters of `split` blocks, which take a share of K each; PAIR:
// of two, which share a tile of 256 rows of P.
template <int TN, bool PAIR, bool PER_Q>
__global__ void __launch_bounds__(Shape<TN, PAIR>::kThreads, Shape<TN, PAIR>::kBlocks)
    kda_fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                          const Fp8MatmulArgs a, const int32_t split) {
    using S = Shape<TN, PAIR>;
    constexpr bool SWAP = !PAIR;  // pairs are for many rows
    static_assert(PAIR || PER_Q, "x's rows, which the few are of, have a scale each");
    static_assert(S::kBlocks * (smem_bytes<TN, PAIR>() + 1024) <= 228 * 1024, "kBlocks of them fit an SM");
    extern __shared__ uint8_t raw[];
    uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    using Sh = Shared<TN, PAIR>;
    Sh& s = *reinterpret_cast<Sh*>(ring + S::kStages * S::kStage);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t half = PAIR ? blockIdx.x & 1 : 0;  // of the pair
    const int32_t rank = !PAIR && split > 1 ? static_cast<int32_t>(blockIdx.x) % split : 0;
    const int32_t together = PAIR ? 2 : split;
    const int32_t first = blockIdx.x / together, step = gridDim.x / together;
    const int32_t KB = (a.K + kFp8Block - 1) / kFp8Block, quads = (KB + kQuad - 1) / kQuad;
    const int32_t k_begin = kQuad * static_cast<int32_t>(static_cast<int64_t>(quads) * rank / (PAIR ? 1 : split));
    const int32_t k_end = min(KB, kQuad * static_cast<int32_t>(static_cast<int64_t>(quads) * (rank + 1) / (PAIR ? 1 : split)));
    const bool p_shared = SWAP && a.w_div != 1;  // the 128 rows of p have one scale
    volatile int32_t* stop = &s.stop;

    if (warp == S::kCopy && lane == 0) {
        prefetch_tmap(&map_p);
        prefetch_tmap(&map_q);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < S::kScaleStages; ++i) {
            mbar_init(&s.scale_full[i], 1);
            mbar_init(&s.scale_empty[i], S::kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.done[i], 1);
            mbar_init(&s.taken[i], S::kWarps * (PAIR ? 2 : 1));
        }
        mbar_init(&s.drained, 1);
        s.stop = 0;
        fence_mbar_init();
    }
    if (warp == S::kMultiply) {
        if constexpr (PAIR) {
            pair_tmem_alloc(&s.tmem, S::kTmem);
        } else {
            tmem_alloc(&s.tmem, S::kTmem);
            tmem_relinquish();
        }
        tc_fence_before();
    }
    if (a.offsets && a.device_status) {  // 0 = o_0 <= ... <= o_E <= rows
        bool ok = true;
        for (int64_t e = static_cast<int64_t>(blockIdx.x) * S::kThreads + threadIdx.x; e <= a.experts;
             e += static_cast<int64_t>(gridDim.x) * S::kThreads) {
            const int32_t o = a.offsets[e];
            ok &= e == 0 ? o == 0 : o >= a.offsets[e - 1];
            ok &= o <= a.rows;
        }
        if (!ok) atomicOr(a.device_status, KDA_DEV_BAD_CU_SEQLENS);
    }
    __syncthreads();
    if (PAIR) cluster_sync();  // the other's barriers are set
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    Walk<TN, PAIR> walk;
    Tile t;
    bool met = false;  // at the cluster's first barrier, behind which its blocks exchange their sums

    if (warp == S::kCopy) {
        // the operands of every block of K, by TMA
        uint32_t it = 0;
        bool going = true;
        for (int32_t tile = first; going && walk.find(a, tile, &t); tile += step) {
            t.p0 += half * kTileP;
            for (int32_t kb = k_begin; kb < k_end; ++kb, ++it) {
                const uint32_t st = it % S::kStages;
                if (!wait_for(&s.empty[st], (it / S::kStages & 1) ^ 1, stop, a.device_status)) {
                    going = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t *at = ring + st * S::kStage, *at_q = at + kTileP * kFp8Block;
                    const int32_t k = kb * kFp8Block;
                    if constexpr (PAIR) {
                        if (half == 0) mbar_arrive_expect_tx(&s.full[st], 2 * S::kStage);
                        const uint32_t bar = cluster_address(smem_u32(&s.full[st]), 0);
                        pair_tma_load_3d(at, &map_p, bar, k, t.p0, 0);
                        pair_tma_load_3d(at_q, &map_q, bar, k, t.q0 + half * S::kQ, t.expert);
                    } else {
                        mbar_arrive_expect_tx(&s.full[st], S::kStage);
                        tma_load_3d(at, &map_p, &s.full[st], k, t.p0, t.expert);
                        tma_load_3d(at_q, &map_q, &s.full[st], k, t.q0, 0);
                    }
                }
                __syncwarp();
            }
        }
        // what was begun has to land before the block ends (a pair's barrier may wait for what the other one did not begin)
        if (*stop && lane == 0 && half == 0)
            for (uint32_t i = it > S::kStages ? it - S::kStages : 0; i < it; ++i)
                (void)mbar_wait(&s.full[i % S::kStages], i / S::kStages & 1, PAIR ? kDrainLimit / 16 : kDrainLimit);
        __syncwarp();
    } else if (warp == S::kScales) {
        // The scales of kQuad blocks of K at a time, 16 bytes of a row, whose rows lie ceil(K / 128) scales apart; q's are turned
        // over, so that the epilogue reads those of four columns at once.
        const float* p_scales = SWAP ? a.w_scales : a.x_scales;
        const float* q_scales = SWAP ? a.x_scales : a.w_scales;
        const int32_t p_div = SWAP ? a.w_div : 1, q_div = SWAP ? 1 : a.w_div;
        const int64_t w_rows = (a.N + a.w_div - 1) / a.w_div;
        const bool whole = KB % kQuad == 0 && ((reinterpret_cast<uintptr_t>(p_scales) | reinterpret_cast<uintptr_t>(q_scales)) & 15) == 0;
        const auto load = [&](const float* row, int32_t kb, bool in) {
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && whole) {
                r = __ldg(reinterpret_cast<const float4*>(row + kb));
            } else if (in) {
                r.x = __ldg(row + kb);
                if (kb + 1 < KB) r.y = __ldg(row + kb + 1);
                if (kb + 2 < KB) r.z = __ldg(row + kb + 2);
                if (kb + 3 < KB) r.w = __ldg(row + kb + 3);
            }
            return r;
        };
        constexpr int kEach = PER_Q ? 1 : kFp8Block, kLoadsQ = (TN / kEach + 31) / 32;  // columns of a scale, loads of a lane
        uint32_t quad = 0;
        bool going = true;
        for (int32_t tile = first; going && walk.find(a, tile, &t); tile += step) {
            const float* ps = p_scales + (SWAP ? t.expert * w_rows : 0) * KB;
            const float* qs = q_scales + (SWAP ? 0 : t.expert * w_rows) * KB;
            const int32_t p_end = SWAP ? a.N : t.row_end, q_end = SWAP ? t.row_end : a.N;
            t.p0 += half * kTileP;
            for (int32_t kb = k_begin; kb < k_end; kb += kQuad, ++quad) {
                float4 p4[kTileP / 32], q4[kLoadsQ];
#pragma unroll
                for (int i = 0; i < kTileP / 32; ++i) {
                    const int32_t p = t.p0 + i * 32 + lane;
                    const bool in = p < p_end && (!p_shared || (i == 0 && lane == 0));
                    p4[i] = load(ps + static_cast<int64_t>(in ? p / p_div : 0) * KB, kb, in);
                }
#pragma unroll
                for (int i = 0; i < kLoadsQ; ++i) {
                    const int32_t q = t.q0 + (i * 32 + lane) * kEach;
                    const bool in = i * 32 + lane < TN / kEach && q < q_end;
                    q4[i] = load(qs + static_cast<int64_t>(in ? q / q_div : 0) * KB, kb, in);
                }
                const uint32_t sc = quad % S::kScaleStages;
                if (!wait_for(&s.scale_empty[sc], (quad / S::kScaleStages & 1) ^ 1, stop, a.device_status)) {
                    going = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kTileP / 32; ++i) *reinterpret_cast<float4*>(s.p_scale[sc][i * 32 + lane]) = p4[i];
#pragma unroll
                for (int i = 0; i < kLoadsQ; ++i) {
                    const int at = i * 32 + lane;
                    if (at >= TN / kEach) break;
                    s.q_scale[sc][0][at] = q4[i].x;
                    s.q_scale[sc][1][at] = q4[i].y;
                    s.q_scale[sc][2][at] = q4[i].z;
                    s.q_scale[sc][3][at] = q4[i].w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.scale_full[sc]);
            }
        }
        __syncwarp();
    } else if (warp == S::kMultiply) {
        // Products, by one lane (of a pair's first block).  The whole warp goes through the loop, so that descriptors and addresses stay in
        // uniform registers: what this warp does for a block has to take less than its 512 cycles, with 16 others that issue beside it.
        constexpr uint32_t idesc = idesc_e4m3(kTileP * (PAIR ? 2 : 1), TN);
        const uint64_t desc = sdesc_sw128(smem_u32(ring), 0, 1024);
        uint32_t st = 0, st_parity = 0, acc = 0, acc_parity = 1;
        bool going = half == 0;
        for (int32_t tile = first; going && walk.find(a, tile, &t); tile += step) {
            for (int32_t kb = k_begin; kb < k_end; ++kb) {
                // the accumulator is what it waits for
                going = wait_for(&s.full[st], st_parity, stop, a.device_status) && wait_for(&s.taken[acc], acc_parity, stop, a.device_status);
                if (!going) break;
                tc_fence_after();
                const uint64_t dp = desc + st * (S::kStage >> 4), dq = dp + (kTileP * kFp8Block >> 4);
                const uint32_t to = tmem + acc * TN;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kFp8Block / 32; ++k) {  // 32 of K are 32 bytes of a row: 2 of the descriptor's 16
                        if constexpr (PAIR) pair_mma_e4m3(to, dp + 2 * k, dq + 2 * k, idesc, k > 0);
                        else mma_e4m3(to, dp + 2 * k, dq + 2 * k, idesc, k > 0);
                    }
                    if constexpr (PAIR) {
                        pair_commit(&s.done[acc]);
                        pair_commit(&s.empty[st]);
                    } else {
                        mma_commit(&s.done[acc]);
                        mma_commit(&s.empty[st]);
                    }
                }
                __syncwarp();
                acc ^= 1;
                acc_parity ^= acc == 0;
                if (++st == S::kStages) {
                    st = 0;
                    st_parity ^= 1;
                }
            }
        }
        if (*stop && half == 0) {
            if (lane == 0) {
                if constexpr (PAIR) pair_commit(&s.drained);
                else mma_commit(&s.drained);
                (void)mbar_wait(&s.drained, 0, kDrainLimit);
            }
            __syncwarp();
        }
    } else {
        // sums over the blocks: a thread has a row p and kCols of the q
        const int quarter = warp & 3, col0 = (warp >> 2) * S::kCols;
        const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
        const int prow = quarter * 32 + lane;
        const uint32_t taken0 = PAIR ? cluster_address(smem_u32(&s.taken[0]), 0) : 0;  // in the pair's first block
        uint32_t acc = 0, acc_parity = 0, sc = 0, sc_parity = 0;
        bool going = true;
        for (int32_t tile = first; going && walk.find(a, tile, &t); tile += step) {
            t.p0 += half * kTileP;
            float sum[S::kCols];
#pragma unroll
            for (int j = 0; j < S::kCols; ++j) sum[j] = 0.f;
            for (int32_t kb = k_begin; kb < k_end; ++kb) {
                const int j4 = kb % kQuad;  // k_begin is a quad's
                if (j4 == 0) {
                    if (!wait_for(&s.scale_full[sc], sc_parity, stop, a.device_status)) {
                        going = false;
                        break;
                    }
                }
                const float* qs = s.q_scale[sc][j4];
                float scale = s.p_scale[sc][p_shared ? 0 : prow][j4];
                if (!PER_Q) scale *= qs[col0 / kFp8Block];
                const uint64_t scale2 = pair_of(scale, scale);
                if (!wait_for(&s.done[acc], acc_parity, stop, a.device_status)) {
                    going = false;
                    break;
                }
                tc_fence_after();
                // The next products may come once all of it is in registers, before the last sums (8192 x 8192 x 4096 243 -> 231 us); not with
                // a scale for every q, whose registers the compiler then moves to memory (409 against 354).
                const auto hand_back = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) cluster_arrive(taken0 + acc * 8);
                        else mbar_arrive(&s.taken[acc]);
                    }
                };
#pragma unroll
                for (int c = 0; c < S::kCols; c += 16) {
                    float v[16];
                    tmem_ld16(from + acc * TN + c, v);
                    tmem_ld_wait16(v);
                    if (!PER_Q && c + 16 == S::kCols) hand_back();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        uint64_t by[2] = {scale2, scale2};
                        if constexpr (PER_Q) {
                            const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qs + col0 + c + j);
                            by[0] = mul2(scale2, q.x);
                            by[1] = mul2(scale2, q.y);
                        }
                        fma2(sum + c + j, v + j, by[0]);
                        fma2(sum + c + j + 2, v + j + 2, by[1]);
                    }
                }
                if (PER_Q) hand_back();
                if (j4 == kQuad - 1 || kb + 1 == k_end) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.scale_empty[sc]);
                    if (++sc == S::kScaleStages) {
                        sc = 0;
                        sc_parity ^= 1;
                    }
                }
                acc ^= 1;
                acc_parity ^= acc == 0;
            }
            if (!going) break;
            const int32_t p = t.p0 + prow;
            if (!PAIR && split > 1) {
                // Each block adds a share of the columns up.  The others' sums of it come into its ring, [rank][column][row], once all are
                // done with theirs: stores that nothing waits for, where loads from the others took a round trip a column.
                cluster_sync();
                const int per = TN / split;  // split divides TN
#pragma unroll
                for (int j = 0; j < S::kCols; ++j) {
                    const int to = (col0 + j) / per, at = rank * per + (col0 + j) % per;
                    cluster_store(cluster_address(smem_u32(ring + (at * kTileP + prow) * 4), to), sum[j]);
                }
                met = true;
                break;
            }
            if (SWAP) {
                if (p < a.N) {
#pragma unroll
                    for (int j = 0; j < S::kCols; ++j)
                        if (t.q0 + col0 + j < t.row_end) store1(a, static_cast<int64_t>(t.q0 + col0 + j) * a.N + p, sum[j]);
                }
            } else {
                // 64 bytes of every row at a time, turned over in shared memory: 4 lanes a row where rows are whole vectors apart, else a lane a
                // column (6418 x 3005 x 1216: 57 us, with a row a lane 234)
                uint8_t* staged = s.staged[warp];
                const int size = a.out_f32 ? 4 : 2;
                const int32_t q0 = t.q0 + col0, row0 = t.p0 + quarter * 32;
                const bool vectors = q0 + S::kCols <= a.N && a.N % 8 == 0;
                const int64_t first_out = static_cast<int64_t>(row0) * a.N + q0;
                const auto turn = [&](int at, int chunk) { return staged + at * S::kStaged + ((chunk ^ (at >> 1)) & 3) * 16; };
                const auto leave = [&](int j) {  // columns j and on
                    __syncwarp();
                    if (vectors) {
                        uint8_t* to = static_cast<uint8_t*>(a.out) + (first_out + j) * size;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = i * 8 + lane / 4;
                            if (row0 + r < t.row_end)
                                *reinterpret_cast<uint4*>(to + static_cast<int64_t>(r) * a.N * size + lane % 4 * 16) =
                                    *reinterpret_cast<const uint4*>(turn(r, lane % 4));
                        }
                    } else if (a.out_f32) {
                        const int c = lane % 16;
                        float* to = static_cast<float*>(a.out) + first_out + j + c;
#pragma unroll 2
                        for (int r = lane / 16; r < 32; r += 2)
                            if (row0 + r < t.row_end && q0 + j + c < a.N)
                                to[static_cast<int64_t>(r) * a.N] = *reinterpret_cast<const float*>(turn(r, c / 4) + c % 4 * 4);
                    } else {
                        uint16_t* to = static_cast<uint16_t*>(a.out) + first_out + j + lane;
#pragma unroll 2
                        for (int r = 0; r < 32; ++r)
                            if (row0 + r < t.row_end && q0 + j + lane < a.N)
                                to[static_cast<int64_t>(r) * a.N] = *reinterpret_cast<const uint16_t*>(turn(r, lane / 8) + lane % 8 * 2);
                    }
                    __syncwarp();
                };
                if (a.out_f32) {
#pragma unroll
                    for (int j = 0; j < S::kCols; j += 16) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<float4*>(turn(lane, i)) = make_float4(sum[j + 4 * i], sum[j + 4 * i + 1], sum[j + 4 * i + 2], sum[j + 4 * i + 3]);
                        leave(j);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < S::kCols; j += 32) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float* v = sum + j + 8 * i;
                            *reinterpret_cast<uint4*>(turn(lane, i)) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                        }
                        leave(j);
                    }
                }
            }
        }
    }
    if (!PAIR && split > 1) {
        if (!met) cluster_sync();
        cluster_sync();
        Walk<TN, PAIR> again;
        if (warp < S::kWarps && !*stop && again.find(a, first, &t)) {
            const int per = TN / split, prow = threadIdx.x % kTileP;
            const int32_t p = t.p0 + prow;
            const float* from = reinterpret_cast<const float*>(ring);
            for (int j = threadIdx.x / kTileP; j < per; j += S::kWarps * 32 / kTileP) {
                float sum = 0.f;
                for (int r = 0; r < split; ++r) sum += from[(r * per + j) * kTileP + prow];  // in the order of K
                const int32_t q = t.q0 + rank * per + j;
                if (p < a.N && q < t.row_end) store1(a, static_cast<int64_t>(q) * a.N + p, sum);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the products of both are done
    if (warp == S::kMultiply) {
        tc_fence_after();
        if constexpr (PAIR) pair_tmem_dealloc(tmem, S::kTmem);
        else tmem_dealloc(tmem, S::kTmem);
    }
}

// Rows of 128 codes of [outer, rows, K], `box` of them, 128-byte swizzled; what lies behind K or the rows reads as zeros.
bool code_map(CUtensorMap* m, const void* base, int32_t K, int32_t rows, int32_t outer, int32_t box) {
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(K) * rows};
    const cuuint32_t sizes[3] = {kFp8Block, static_cast<cuuint32_t>(box), 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, sizes, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, bool PAIR, bool PER_Q>
cudaError_t launch(const Fp8MatmulArgs& a, int split, int64_t tiles, cudaStream_t stream) {
    using S = Shape<TN, PAIR>;
    static int configured[64] = {};
    CUtensorMap map_p, map_q;
    if (!(PAIR ? code_map(&map_p, a.x, a.K, a.rows, 1, kTileP) && code_map(&map_q, a.w, a.K, a.N, a.experts, S::kQ)
               : code_map(&map_p, a.w, a.K, a.N, a.experts, kTileP) && code_map(&map_q, a.x, a.K, a.rows, 1, TN)))
        return cudaErrorUnknown;
    const auto kernel = kda_fp8_matmul_kernel<TN, PAIR, PER_Q>;
    constexpr uint32_t smem = smem_bytes<TN, PAIR>();
    const cudaError_t err = set_smem(kernel, smem, configured);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    const int64_t most = static_cast<int64_t>(device_sm_count()) * S::kBlocks;
    cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? 2 * std::min(tiles, most / 2) : split > 1 ? tiles * split : std::min(tiles, most)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR || split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, map_p, map_q, a, static_cast<int32_t>(split));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of TN rows of x by 128 of w; with a clusters' blocks on shares of K while they find places.
int64_t few_tiles(const Fp8MatmulArgs& a, int TN) {
    // of experts at most so many: one's last tile is not whole
    return (a.offsets ? std::min<int64_t>(a.rows, a.rows / TN + a.experts) : ceil_div(a.rows, TN)) * ceil_div(a.N, kTileP);
}
template <int TN>
int64_t places() {
    return static_cast<int64_t>(device_sm_count()) * Shape<TN, false>::kBlocks;
}
template <int TN>
cudaError_t few_rows(const Fp8MatmulArgs& a, cudaStream_t stream) {
    const int64_t tiles = few_tiles(a, TN), quads = ceil_div(a.K, kFp8Block * kQuad);
    int split = 1;
    if (!a.offsets)
        while (split < kMaxSplit && tiles * split * 2 <= places<TN>() && split * 2 <= quads) split *= 2;
    return launch<TN, false, true>(a, split, tiles, stream);
}
cudaError_t many_rows(const Fp8MatmulArgs& a, cudaStream_t stream) {
    constexpr int kPair = 2 * kTileP;
    const int64_t tiles = (a.offsets ? a.rows / kPair + a.experts : ceil_div(a.rows, kPair)) * ceil_div(a.N, 256);
    return a.w_div == 1 ? launch<256, true, true>(a, 1, tiles, stream) : launch<256, true, false>(a, 1, tiles, stream);
}

}  // namespace

// Few rows: as small a tile as gives every tile a place at once, since a block's time is a chain of K blocks that grows with the tile;
// then pairs, whose tiles are the most per byte.  Of experts' rows, which the host knows the average of, the tile that holds that.
// (us with K = 4096, tiles of 16, 32, 64, 128 rows, pairs of 256:
//     24 x 4096: 15.5  17.5  19.6  21.6  25.7       128 x 2048: 19.6  17.5  19.6  29.8  27.8
//    128 x 8192: 31.9  22.7  27.8  26.8  27.8       256 x 4096: 31.9  22.7  27.8  25.7  27.7
//    256 x 8192: 50.3  33.9  27.8  24.7  27.8       512 x 4096: 49.3  32.9  27.8  23.7  27.8
//    384 x 8192: 70.8  45.2  42.1  39.0  27.8      1024 x 4096: 82.1  53.4  46.2  39.0  27.8
//  32 experts of 2048 x 2048, rows in all:    512:  38.0  37.0  38.0  44.2  48.3      1024: 43.2  38.0  38.0  45.2  50.3
//                                            2048:  55.5  45.2  42.1  44.2  50.3      4096: 91.3  61.6  57.5  58.5  52.4)
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    if (a.offsets) {
        const int64_t each = ceil_div(a.rows, a.experts);
        return each <= 8 ? few_rows<16>(a, stream) : each <= 32 ? few_rows<32>(a, stream) : each <= 80 ? few_rows<64>(a, stream) : many_rows(a, stream);
    }
    if (a.rows <= 24) return few_rows<16>(a, stream);
    if (few_tiles(a, 32) <= places<32>()) return few_rows<32>(a, stream);
    return few_tiles(a, 128) <= places<128>() ? few_rows<128>(a, stream) : many_rows(a, stream);
}

}  // namespace kda
