// glu.cu -- the gated feed-forward block's kernels: both projections, the activation,
// the product and its quantize in one GEMM (fp8_glu_fwd), and the gradient of that in
// the down-projection's dgrad (fp8_gemm_dgrad_glu).
//
//   forward   [g | u] = X W1 (E4M3 x E4M3, FP32 sums); a = act(g) u; q = E4M3(BF16(a) s)
//   backward  dA = dY W2^T (E5M2 x E4M3, FP32 sums); dg = dA u act'(g), du = dA act(g)
//
// Both are the tcgen05 GEMM D[M, .] = A[M,K] . B[., K]^T of gemm_parts.cuh's pieces with
// an epilogue of their own.  A CTA is 10 warps (backward 18), persistent over output tiles:
//   warp 0     TMA producer: k-blocks of 128 bytes a row into a ring of stages
//   warp 1     MMA issuer: kind::f8f6f4 into one of two TMEM accumulators
//   the others epilogue: two (backward four) warps a TMEM lane quarter, 32-column chunks in turn
// PAIR: a cluster of two CTAs, 256 rows a tile, cta_group::2.
//
// The forward tile of BN accumulator columns is BN / 2 columns of the gate and the same
// BN / 2 of the up-projection side by side, so that a thread holds g and u of one element
// and nothing but the product leaves the SM.  In a pair each CTA loads one of the two as
// its half of B: the MMA reads B's first half from the leader's shared memory (the gate's
// rows of W1^T) and its second from the peer's (the up-projection's).
//
// The epilogue is a thread a row, 32 columns (a chunk) at a time, and stores without shared
// memory: 32 bytes of a thread's own row, a whole sector each, and the transposed codes after
// exchanges between lanes.  No fence or copy engine stands between the accumulator and memory,
// and the operands' ring has the shared memory that staging would take.  The backward's chunks
// of g and u come by TMA into a buffer a warp, the next one asked for as soon as this one is in
// registers (32-byte loads straight into registers, 32 sectors an instruction, took 680 us).
//
// What bounds it (GB300).  32768 x 1600 -> 6400 forward with h_out and both code layouts 471 to 490 us, 2.8
// PFLOP/s (one code layout alone 400 us, 3.36; the plain GEMM of the same product 423): busiest are the L1-to-L2
// request path (69 % at 8192 rows) and the tensor pipe (68 % of its cycles), so neither is a limit yet;
// sustained for half a second the 1400 W cap holds the SMs at 1470 MHz and it takes 540 to 566.  Backward with
// both code layouts 389 to 393 us (GELU 415), 4.4 TB/s: neither memory (DRAM at 44 % of its peak at 8192 rows) nor
// the tensor pipe (37 %); instructions, 18 an element of dA, issue in 46 % of the cycles from at most 4.5 warps a
// scheduler, and the 96 registers that 18 warps leave a thread spill 48 bytes.  A few tokens (1 to 128 x 1600 -> 6400, 20.5 MB of
// weights): 7.5 us with the clearing launch, 13 k-blocks one after another in each of 100 CTAs.
// Not kept: h_out through shared memory in 64-column boxes (508 us: two ring stages less), adjacent instead of
// alternate chunks a warp (backward 417), a kernel of dot products for one or two rows (7.6 and 9.8).
//
// Every wait is bounded as in gemm.cu: on time-out the CTA sets FP8Q_DEV_TIMEOUT, lets its
// copies and MMAs land (bounded), frees TMEM and exits.
#include "common.cuh"
#include "gemm_parts.cuh"
#include "glu_ops.cuh"
#include "norm_ops.cuh"
#include "quant_ops.cuh"
#include "../../include/fp8q_testing.h"

#include <algorithm>
#include <atomic>

namespace fp8q {

namespace {

constexpr int kBoxBytes = 32 * 32 * 2;  // 32 rows x 32 BF16 columns, in the 64-byte swizzle

// Operands; h0 / h1 (backward): the halves of h, each a tensor of its own width, so that a box
// at a half's ragged end is clipped there.
struct GluMaps {
    CUtensorMap a, b, h0, h1;
};

// The tensors of a call.  Forward: x [M,K], w [2F,K], o = h_out [M,2F], d = act_out [M,F], q [M,F], t [F,M].
// Backward: x = dY [M,K], w = W2 [F,K], h [M,2F], o = dh [M,2F], q [M,2F], t [2F,M].
struct GluArgs {
    const void* x;
    const void* w;
    const uint16_t* h;
    uint16_t* o;
    uint16_t* d;
    uint8_t* q;
    uint8_t* t;
    const float* scale_a;
    const float* scale_b;
    const float* scale_q;
    float* amax;
    unsigned long long* sat;
    int* status;
    int64_t M, F, K;
    uint32_t idesc;
    int act;
    bool hold;         // test hook: no operand is loaded, so that the first wait runs out
    uint32_t a_bytes;  // of a CTA's box of A: of a call of less than 128 rows the rows that there are
    bool wide_bf, wide_q;  // every 16 columns of h, o and d (32 of q) of a row are one 32-byte sector
};

template <int BN, bool PAIR, bool BWD>
struct GluCfg {
    static constexpr int OUT = BWD ? BN : BN / 2;       // columns of F a tile covers
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;   // rows of B a CTA loads
    static constexpr int B_BOX = BWD ? B_ROWS : BN / 2; // rows of a TMA box of B
    static constexpr int A_BYTES = BM * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_ROWS * BK;
    static constexpr int TX_BYTES = STAGE_BYTES * (PAIR ? 2 : 1);
    static constexpr int ACCS = 2;
    // epilogue warps: the backward's instructions, twice the forward's, want all that 96 registers a
    // thread allow (32768 x 1600 -> 6400: 385 us with 16, 400 with 12, 453 with 8; forward 476, 483, 483)
    static constexpr int WARPS = BWD ? 16 : 8;
    static constexpr int THREADS = 64 + 32 * WARPS;
    static constexpr int LOADS = BWD ? 1 : 0;           // backward: a warp's buffers for a chunk of g and u
    static constexpr int LOAD_BYTES = WARPS * LOADS * 2 * kBoxBytes;
    static constexpr int BAR_BYTES = 512;
    static constexpr int RING = 232448 - 512 - BAR_BYTES - 1024 - LOAD_BYTES;
    static constexpr int STAGES = RING / STAGE_BYTES < 8 ? RING / STAGE_BYTES : 8;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + LOAD_BYTES + BAR_BYTES + 1024;
    static constexpr int TMEM_COLS = 2 * BN <= 64 ? 64 : 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
    static constexpr int TILE_M = PAIR ? 2 * BM : BM;
    static constexpr int CHUNKS = OUT / 32;
    static_assert(OUT % 32 == 0 && BN <= 256 && STAGES >= 2 && (B_ROWS * BK) % 1024 == 0, "tile shape");
    static_assert((2 * STAGES + 2 * ACCS + 1 + LOADS * WARPS) * 8 + 16 <= BAR_BYTES, "barrier area");
};

// 32 bytes of a thread's row: one access where the row's sectors allow it, else two of 16.
__device__ __forceinline__ void st_32(void* to, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     :: "l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    } else {
        st_v4(to, make_uint4(v[0], v[1], v[2], v[3]));
        st_v4(static_cast<uint8_t*>(to) + 16, make_uint4(v[4], v[5], v[6], v[7]));
    }
}
// The larger magnitudes of two pairs of BF16 values; a NaN stays one.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.NaN.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 columns of this lane's row (packed BF16): their codes in four words, the magnitudes and
// saturations counted.
template <int FMT>
__device__ __forceinline__ void glu_codes(const uint32_t (&v)[8], float s, uint32_t* q, uint32_t& amax2, uint32_t& nsat) {
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) all = max_abs_bf16x2(all, v[j]);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const uint2 c = cast8_codes<FMT>(make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]), s);
        q[2 * g] = c.x;
        q[2 * g + 1] = c.y;
    }
    amax2 = max_abs_bf16x2(amax2, all);
    if (!(__fmul_rn(__uint_as_float(max16x2(all) << 16), s) <= fp8_max_value(FMT))) {  // (a NaN counts the others too)
#pragma unroll
        for (int g = 0; g < 2; ++g)
            nsat += sat_count8<FMT>(make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]), s);
    }
}

// Values of rows behind M or columns behind F, whatever an accumulator holds there (other rows' sums, or an
// infinity times the zeros that fill a box): nothing for the maximum and the count.
__device__ __forceinline__ void none(uint32_t (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0;
}

// The magnitudes alone (a call that wants a maximum but no codes).
__device__ __forceinline__ void glu_amax(const uint32_t (&v)[8], uint32_t& amax2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) amax2 = max_abs_bf16x2(amax2, v[j]);
}

// Codes of W words (4 W columns) of 32 rows to the transposed tensor [., M], whose row `col` is at
// `to` (this lane's piece of 4 rows).  Four lanes turn 4 x 4 bytes by two exchanges: neighbouring
// lanes swap odd for even bytes, then pairs of lanes high for low halves; lane 4 k + i then holds
// rows 4 k .. 4 k + 3 of column 4 w + i, and a warp's store is four whole 32-byte sectors.
template <int W>
__device__ __forceinline__ void glu_turned(const uint32_t* q, uint8_t* to, int64_t M, int lane, bool in) {
    const uint32_t sel1 = lane & 1 ? 0x3715u : 0x6240u, sel2 = lane & 2 ? 0x3276u : 0x5410u;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t x = __byte_perm(q[w], __shfl_xor_sync(0xFFFFFFFFu, q[w], 1), sel1);
        x = __byte_perm(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2), sel2);
        if (in) *reinterpret_cast<uint32_t*>(to) = x;
        to += 4 * M;
    }
}

__device__ __forceinline__ f32x2 acc_pair(uint32_t a, uint32_t b) { return pair_of(__uint_as_float(a), __uint_as_float(b)); }

// 16 accumulator columns each of g and u -> packed BF16 a.
template <int ACT>
__device__ __forceinline__ void glu_products(const uint32_t (&g)[16], const uint32_t (&u)[16], float inv, uint32_t (&a)[8]) {
    const f32x2 inv2 = twice(inv);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        a[j] = bf16x2_of(mul2(glu_act<ACT>(mul2(acc_pair(g[2 * j], g[2 * j + 1]), inv2)),
                              mul2(acc_pair(u[2 * j], u[2 * j + 1]), inv2)));
}

// The accumulator's columns as packed BF16.
__device__ __forceinline__ void glu_stored(const uint32_t (&r)[16], float inv, uint32_t (&h)[8]) {
    const f32x2 inv2 = twice(inv);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = bf16x2_of(mul2(acc_pair(r[2 * j], r[2 * j + 1]), inv2));
}

// 16 columns of dA, g and u -> packed BF16 dg and du.
template <int ACT>
__device__ __forceinline__ void glu_gradients(const uint32_t (&r)[16], float inv, const uint32_t (&g)[8],
                                              const uint32_t (&u)[8], uint32_t (&dg)[8], uint32_t (&du)[8]) {
    const f32x2 inv2 = twice(inv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const f32x2 d = mul2(acc_pair(r[2 * j], r[2 * j + 1]), inv2);
        f32x2 f, slope;
        glu_act_grad<ACT>(f32x2_of(g[j]), f, slope);
        dg[j] = bf16x2_of(mul2(mul2(d, f32x2_of(u[j])), slope));
        du[j] = bf16x2_of(mul2(d, f));
    }
}

// Arrive on an mbarrier of the cluster without ordering this thread's memory accesses: what the
// arrival reports is that TMEM was read into registers, which the load's own wait has seen to.  (With
// .release it waited until the warp's stores had reached memory, once a tile: of 16 384 x 6400 x 1600
// backward a sixth of the epilogue's stalls.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}

// Two loads of 32 lanes x 16 columns in flight, then one wait.
__device__ __forceinline__ void tmem_ld_2x16_sync(uint32_t taddr0, uint32_t taddr1, uint32_t (&r0)[16], uint32_t (&r1)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r0[0]), "=r"(r0[1]), "=r"(r0[2]), "=r"(r0[3]), "=r"(r0[4]), "=r"(r0[5]), "=r"(r0[6]), "=r"(r0[7]), "=r"(r0[8]), "=r"(r0[9]), "=r"(r0[10]), "=r"(r0[11]), "=r"(r0[12]), "=r"(r0[13]), "=r"(r0[14]), "=r"(r0[15]),
          "=r"(r1[0]), "=r"(r1[1]), "=r"(r1[2]), "=r"(r1[3]), "=r"(r1[4]), "=r"(r1[5]), "=r"(r1[6]), "=r"(r1[7]), "=r"(r1[8]), "=r"(r1[9]), "=r"(r1[10]), "=r"(r1[11]), "=r"(r1[12]), "=r"(r1[13]), "=r"(r1[14]), "=r"(r1[15])
        : "r"(taddr0), "r"(taddr1) : "memory");
}

// The tiles of one CTA (pair), n fastest, without a division a tile.
struct TileWalk {
    int64_t left, m, n, num_n, step, step_m, step_n;  // tiles from here to the last; this one's row and column block
    __device__ __forceinline__ TileWalk(int64_t first, int64_t stride, int64_t tiles, int64_t columns)
        : left(tiles - first), m(first / columns), n(first % columns), num_n(columns), step(stride),
          step_m(stride / columns), step_n(stride % columns) {}
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next() {
        left -= step;
        m += step_m;
        n += step_n;
        if (n >= num_n) {
            n -= num_n;
            ++m;
        }
    }
};

template <int BN, bool PAIR, bool BWD>
__global__ void __launch_bounds__((GluCfg<BN, PAIR, BWD>::THREADS), 1)
glu_kernel(const __grid_constant__ GluMaps maps, const GluArgs p) {
    using C = GluCfg<BN, PAIR, BWD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* boxes = smem + C::STAGES * C::STAGE_BYTES;  // 1024-aligned
    uint64_t* bars = reinterpret_cast<uint64_t*>(boxes + C::LOAD_BYTES);
    uint64_t* full = bars;
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* tempty = tfull + C::ACCS;
    uint64_t* drain = tempty + C::ACCS;
    uint64_t* loaded = drain + 1;  // backward: [warp][buffer]
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(loaded + C::LOADS * C::WARPS);
    volatile int* abort_flag = reinterpret_cast<int*>(tmem_holder) + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int64_t num_n = (p.F + C::OUT - 1) / C::OUT;
    const int64_t num_tiles = ((p.M + C::TILE_M - 1) / C::TILE_M) * num_n;
    TileWalk tile(PAIR ? blockIdx.x / 2 : blockIdx.x, PAIR ? gridDim.x / 2 : gridDim.x, num_tiles, num_n);
    const int num_kb = static_cast<int>((p.K + BK - 1) / BK);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < C::ACCS; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), C::WARPS * (PAIR ? 2 : 1));
        }
        mbar_init(smem_u32(drain), 1);
        for (int i = 0; i < C::LOADS * C::WARPS; ++i) mbar_init(smem_u32(&loaded[i]), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_holder), C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the peer's barriers exist before any copy signals them
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_launch_dependents();
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (; tile.more() && ok && !p.hold; tile.next()) {
                const int32_t m0 = static_cast<int32_t>(tile.m * C::TILE_M + rank * BM);
                const int32_t n0 = static_cast<int32_t>(tile.n * C::OUT);
                const int32_t up = static_cast<int32_t>(p.F) + n0;  // forward: the up-projection's rows of W1^T
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!wait_phase(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES), sb = sa + C::A_BYTES;
                    if constexpr (PAIR) {
                        const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
                        if (leader) mbar_arrive_expect_tx(smem_u32(&full[stage]), C::TX_BYTES);
                        tma_load_2d_pair(sa, &maps.a, fb, kb * BK, m0);
                        const int32_t row = BWD ? n0 + static_cast<int32_t>(rank) * C::B_ROWS : leader ? n0 : up;
                        tma_load_2d_pair(sb, &maps.b, fb, kb * BK, row);
                    } else {
                        const uint32_t fb = smem_u32(&full[stage]);
                        mbar_arrive_expect_tx(fb, C::TX_BYTES - C::A_BYTES + p.a_bytes);
                        tma_load_2d(sa, &maps.a, fb, kb * BK, m0);
                        tma_load_2d(sb, &maps.b, fb, kb * BK, n0);
                        if constexpr (!BWD) tma_load_2d(sb + C::B_BOX * BK, &maps.b, fb, kb * BK, up);
                    }
                    ++issued;
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // no copy may still be landing in shared memory when the CTA exits
            if (!PAIR || leader) {
                const int64_t tail = issued < C::STAGES ? issued : C::STAGES;
                for (int64_t j = 1; j <= tail; ++j) {
                    int s = stage - static_cast<int>(j);
                    uint32_t ph = phase;
                    if (s < 0) { s += C::STAGES; ph ^= 1u; }
                    wait_phase_drain(&full[s], ph);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (; tile.more() && ok; tile.next()) {
                if (!wait_phase(&tempty[acc], acc_phase ^ 1u, abort_flag, p.status)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!wait_phase(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + stage * C::STAGE_BYTES), b_addr = a_addr + C::A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k) {
                        const uint64_t ad = smem_desc_k_sw128(a_addr + k * UMMA_K), bd = smem_desc_k_sw128(b_addr + k * UMMA_K);
                        if constexpr (PAIR) mma_f8f6f4_pair(d_tmem, ad, bd, p.idesc, kb > 0 || k > 0);
                        else mma_f8f6f4(d_tmem, ad, bd, p.idesc, kb > 0 || k > 0);
                    }
                    if constexpr (PAIR) mma_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
                    else mma_commit(smem_u32(&empty[stage]));
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                if constexpr (PAIR) mma_commit_pair_mc(smem_u32(&tfull[acc]), 0x3);
                else mma_commit(smem_u32(&tfull[acc]));
                next_acc<C::ACCS>(acc, acc_phase);
            }
            // all MMAs of this thread complete before TMEM is released
            if constexpr (PAIR) mma_commit_pair(smem_u32(drain));
            else mma_commit(smem_u32(drain));
            wait_phase_drain(drain, 0);
        }
    } else {
        constexpr int STEP = C::WARPS / 4;
        const int quarter = warp & 3;     // TMEM lane quarter of this warp
        const int c0 = (warp - 2) / 4;    // its first chunk, and every STEPth one from there
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : smem_u32(&tempty[0]);
        const float inv = 1.0f / (__ldg(p.scale_a) * __ldg(p.scale_b));
        const float s_q = p.scale_q ? __ldg(p.scale_q) : 0.0f;
        uint32_t amax2 = 0, nsat = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool arrived = true;

        const int64_t row_in_tile = rank * BM + quarter * 32 + lane;
        auto row_of = [&](const TileWalk& w) { return w.m * C::TILE_M + row_in_tile; };
        auto col_of = [&](const TileWalk& w, int c) { return w.n * C::OUT + c * 32; };

        // backward: this warp's chunks of g and u, in the order in which they are used; `asked` of them
        // are on the way or read, `used` of them read
        constexpr int LOADS = C::LOADS > 0 ? C::LOADS : 1;
        uint8_t* const box0 = boxes + (warp - 2) * C::LOADS * 2 * kBoxBytes;
        uint64_t* const bar = loaded + C::LOADS * (warp - 2);
        TileWalk ask_tile = tile;
        int ask_c = c0;
        uint32_t asked = 0, used = 0;
        auto ask = [&]() {
            while (ask_tile.more() && (ask_c >= C::CHUNKS || row_of(ask_tile) - lane >= p.M || col_of(ask_tile, ask_c) >= p.F)) {
                ask_tile.next();
                ask_c = c0;
            }
            if (!ask_tile.more()) return;
            if (lane == 0) {
                const uint32_t b = smem_u32(&bar[asked % LOADS]), to = smem_u32(box0 + (asked % LOADS) * 2 * kBoxBytes);
                const int32_t x = static_cast<int32_t>(col_of(ask_tile, ask_c)), y = static_cast<int32_t>(row_of(ask_tile));
                mbar_arrive_expect_tx(b, 2 * kBoxBytes);
                tma_load_2d(to, &maps.h0, b, x, y);
                tma_load_2d(to + kBoxBytes, &maps.h1, b, x, y);
            }
            ++asked;
            ask_c += STEP;
        };
        if constexpr (BWD) {
            for (int i = 0; i < LOADS; ++i) ask();
        }

        for (; tile.more(); tile.next()) {
            const int64_t row = row_of(tile);
            const bool in = row < p.M;
            if (!__all_sync(0xFFFFFFFFu, wait_phase(&tfull[acc], acc_phase, abort_flag, p.status))) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + lane_base + static_cast<uint32_t>(acc * BN);
            // this lane's part of the transposed codes: rows 4 (lane / 4) .. + 3 of the warp's 32, column lane % 4
            const int64_t trow = row - lane + (lane >> 2) * 4;
            const bool tin = trow < p.M;
            bool released = false;
            auto release = [&]() {  // this warp's columns of the accumulator are in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster_relaxed(tempty0 + 8u * acc);
                    else mbar_arrive(tempty0 + 8u * acc);
                }
                released = true;
            };
#pragma unroll 1
            for (int c = c0; c < C::CHUNKS; c += STEP) {
                const int64_t col0 = col_of(tile, c);
                if (row - lane >= p.M || col0 >= p.F) break;
                const bool whole = col0 + 32 <= p.F;  // otherwise F ends after 16 columns
                const bool last = c + STEP >= C::CHUNKS || col0 + STEP * 32 >= p.F;
                uint32_t q[BWD ? 2 : 1][8];
                const uint8_t* box = box0 + (used % LOADS) * 2 * kBoxBytes + lane * 64;
                if constexpr (BWD) {
                    arrived = __all_sync(0xFFFFFFFFu, wait_phase(&bar[used % LOADS], (used / LOADS) & 1, abort_flag, p.status));
                    if (!arrived) break;
                    ++used;
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int64_t col = col0 + half * 16;
                    const bool ok = in && (half == 0 || whole);
                    if constexpr (!BWD) {
                        uint32_t g[16], u[16], a[8];
                        tmem_ld_2x16_sync(taddr + c * 32 + half * 16, taddr + C::OUT + c * 32 + half * 16, g, u);
                        if (half == 1 && last) release();
                        switch (p.act) {
                            case FP8Q_ACT_IDENTITY: glu_products<FP8Q_ACT_IDENTITY>(g, u, inv, a); break;
                            case FP8Q_ACT_RELU: glu_products<FP8Q_ACT_RELU>(g, u, inv, a); break;
                            case FP8Q_ACT_RELU2: glu_products<FP8Q_ACT_RELU2>(g, u, inv, a); break;
                            case FP8Q_ACT_SILU: glu_products<FP8Q_ACT_SILU>(g, u, inv, a); break;
                            default: glu_products<FP8Q_ACT_GELU>(g, u, inv, a); break;
                        }
                        if (!ok) none(a);
                        if (p.o) {
                            uint32_t hv[8];
                            uint16_t* at = p.o + row * 2 * p.F + col;
                            glu_stored(g, inv, hv);
                            if (ok) st_32(at, hv, p.wide_bf);
                            glu_stored(u, inv, hv);
                            if (ok) st_32(at + p.F, hv, p.wide_bf);
                        }
                        if (p.d && ok) st_32(p.d + row * p.F + col, a, p.wide_bf);
                        if (p.scale_q) glu_codes<FP8Q_E4M3>(a, s_q, &q[0][half * 4], amax2, nsat);
                        else glu_amax(a, amax2);
                    } else {
                        uint32_t r[16], g[8], u[8], dg[8], du[8];
                        tmem_ld_x16_sync(taddr + c * 32 + half * 16, r);
                        if (half == 1 && last) release();
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int at = ((2 * half + k) ^ ((lane >> 1) & 3)) << 4;
                            const uint4 g4 = *reinterpret_cast<const uint4*>(box + at), u4 = *reinterpret_cast<const uint4*>(box + kBoxBytes + at);
                            g[4 * k] = g4.x; g[4 * k + 1] = g4.y; g[4 * k + 2] = g4.z; g[4 * k + 3] = g4.w;
                            u[4 * k] = u4.x; u[4 * k + 1] = u4.y; u[4 * k + 2] = u4.z; u[4 * k + 3] = u4.w;
                        }
                        if (half == 1) {  // every lane has read its g and u: the buffer takes another chunk
                            __syncwarp();
                            ask();
                        }
                        switch (p.act) {
                            case FP8Q_ACT_IDENTITY: glu_gradients<FP8Q_ACT_IDENTITY>(r, inv, g, u, dg, du); break;
                            case FP8Q_ACT_RELU: glu_gradients<FP8Q_ACT_RELU>(r, inv, g, u, dg, du); break;
                            case FP8Q_ACT_RELU2: glu_gradients<FP8Q_ACT_RELU2>(r, inv, g, u, dg, du); break;
                            case FP8Q_ACT_SILU: glu_gradients<FP8Q_ACT_SILU>(r, inv, g, u, dg, du); break;
                            default: glu_gradients<FP8Q_ACT_GELU>(r, inv, g, u, dg, du); break;
                        }
                        if (!ok) {
                            none(dg);
                            none(du);
                        }
                        if (p.o && ok) {
                            uint16_t* at = p.o + row * 2 * p.F + col;
                            st_32(at, dg, p.wide_bf);
                            st_32(at + p.F, du, p.wide_bf);
                        }
                        if (p.scale_q) {
                            glu_codes<FP8Q_E5M2>(dg, s_q, &q[0][half * 4], amax2, nsat);
                            glu_codes<FP8Q_E5M2>(du, s_q, &q[BWD ? 1 : 0][half * 4], amax2, nsat);
                        } else {
                            glu_amax(dg, amax2);
                            glu_amax(du, amax2);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < (BWD ? 2 : 1); ++k) {
                    const int64_t col = col0 + k * p.F;
                    if (p.q && in) {
                        uint8_t* at = p.q + row * (BWD ? 2 : 1) * p.F + col;
                        if (whole) st_32(at, q[k], p.wide_q);
                        else st_v4(at, make_uint4(q[k][0], q[k][1], q[k][2], q[k][3]));
                    }
                    if (p.t) {
                        uint8_t* at = p.t + (col + (lane & 3)) * p.M + trow;
                        glu_turned<4>(q[k], at, p.M, lane, tin);
                        if (whole) glu_turned<4>(q[k] + 4, at + 16 * p.M, p.M, lane, tin);
                    }
                }
            }
            if (!arrived) break;
            if (!released) release();  // none of the tile is this warp's
            next_acc<C::ACCS>(acc, acc_phase);
        }
        // no load may still be landing in shared memory when the CTA exits
        for (; BWD && used < asked; ++used) wait_phase_drain(&bar[used % LOADS], (used / LOADS) & 1);
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max16x2(amax2));
        const uint32_t n = __reduce_add_sync(0xFFFFFFFFu, nsat);
        if (lane == 0) {
            if (p.amax && m) atomicMax(reinterpret_cast<unsigned int*>(p.amax), m << 16);
            if (p.sat && n) atomicAdd(p.sat, static_cast<unsigned long long>(n));
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the leader's MMAs into both CTAs are done
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------- host --
// A half of h [M,2F]: 32 x 32 boxes in the 64-byte swizzle.
bool make_half_map(CUtensorMap* map, const void* base, int64_t M, int64_t F) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(F), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(4 * F)};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool PAIR, bool BWD>
int launch_glu(GluArgs p, cudaStream_t stream) {
    using C = GluCfg<BN, PAIR, BWD>;
    const auto kern = glu_kernel<BN, PAIR, BWD>;
    // co-resident CTAs (pairs) of the current device, whose copy of the kernel may take the shared memory
    static DeviceTable<1> table;
    int device = 0, units = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return FP8Q_ERR_CUDA;
    const cudaError_t e = table.get(device, 0, &units, [&](int* n) {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (err != cudaSuccess) return err;
        if (!PAIR) {
            *n = sm_count();
            return cudaSuccess;
        }
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2 * sm_count());
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(n, kern, &cfg);
    });
    if (e != cudaSuccess || units < 1) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    const int64_t M = p.M, F = p.F;
    alignas(64) GluMaps maps;
    // a call of fewer rows than a tile copies those alone, to whole swizzle atoms (16 x 1600 -> 6400: filling the
    // other rows with zeros took 3 us of 11); what the other rows' accumulators hold is not used
    const int a_rows = !PAIR && M < BM ? static_cast<int>((M + 7) / 8 * 8) : BM;
    p.a_bytes = static_cast<uint32_t>(a_rows * BK);
    if (!make_kmajor_map(&maps.a, p.x, M, p.K, a_rows) || !make_kmajor_map(&maps.b, p.w, BWD ? F : 2 * F, p.K, C::B_BOX))
        return FP8Q_ERR_CUDA;
    maps.h0 = maps.h1 = maps.a;
    if (BWD && (!make_half_map(&maps.h0, p.h, M, F) || !make_half_map(&maps.h1, p.h + F, M, F))) return FP8Q_ERR_CUDA;
    p.idesc = idesc_f8(BWD ? FP8Q_E5M2 : FP8Q_E4M3, FP8Q_E4M3, C::TILE_M, BN);
    const int64_t tiles = ((M + C::TILE_M - 1) / C::TILE_M) * ((F + C::OUT - 1) / C::OUT);
    const int n = static_cast<int>(std::min<int64_t>(tiles, units));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(PAIR ? 2 * n : n);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, maps, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

// The tile: the one of the least estimated time  c + waves (e + m K / 1000)  in us, where waves are
// the tiles over the CTAs (pairs) that run at a time, rounded up; c, e and m are fits to the seven
// tiles' times over nine shapes a direction (128 to 16384 rows, 256 x 1024 to 1600 x 6400; within 15 %
// each).  A tile's time depends on its width less than on K, and wide tiles lose more to a last wave that
// is not full: 8192 x 768 -> 2048 backward is 38 us in 128-wide pair tiles, 42 in 256-wide ones; 8192 x
// 1600 -> 6400 109 in 256-wide ones and 125 in 128.
std::atomic<int> g_glu_tile{-1};  // fp8q_glu_set_tile: -1 = by the estimate, else (pair << 16) | bn

template <bool BWD>
int dispatch_glu(const GluArgs& p, cudaStream_t stream) {
    struct Cand { bool pair; int bn; double c, e, m; };
    static constexpr Cand kForward[] = {{true, 256, 3.99, 3.72, 1.22}, {true, 192, 4.56, 2.64, 1.25}, {true, 128, 3.85, 1.33, 1.64},
                                        {false, 256, 3.87, 3.37, 2.23}, {false, 192, 4.14, 2.42, 1.93},
                                        {false, 128, 3.76, 1.46, 1.68}, {false, 64, 3.37, 0.73, 1.90}};
    static constexpr Cand kBackward[] = {{true, 256, 7.55, 7.36, 1.35}, {true, 192, 7.34, 5.83, 1.08}, {true, 128, 5.64, 3.76, 1.16},
                                         {false, 256, 6.91, 6.97, 1.99}, {false, 192, 6.22, 6.41, 1.47},
                                         {false, 128, 4.88, 4.35, 0.98}, {false, 64, 4.12, 2.73, 1.15}};
    const int64_t sms = sm_count();
    Cand best = (BWD ? kBackward : kForward)[5];
    double best_cost = -1.0;
    for (const Cand& c : BWD ? kBackward : kForward) {
        if (c.pair && p.M <= BM) continue;
        const int64_t tile_m = c.pair ? 2 * BM : BM, units = c.pair ? sms / 2 : sms, out = BWD ? c.bn : c.bn / 2;
        const int64_t tiles = ((p.M + tile_m - 1) / tile_m) * ((p.F + out - 1) / out);
        const double cost = c.c + static_cast<double>((tiles + units - 1) / units) * (c.e + c.m * 1e-3 * static_cast<double>(p.K));
        if (g_glu_tile.load(std::memory_order_relaxed) == ((c.pair ? 1 << 16 : 0) | c.bn)) { best = c; break; }
        if (best_cost < 0 || cost < best_cost) { best_cost = cost; best = c; }
    }
    if (best.pair) {
        if (best.bn == 256) return launch_glu<256, true, BWD>(p, stream);
        if (best.bn == 192) return launch_glu<192, true, BWD>(p, stream);
        return launch_glu<128, true, BWD>(p, stream);
    }
    if (best.bn == 256) return launch_glu<256, false, BWD>(p, stream);
    if (best.bn == 192) return launch_glu<192, false, BWD>(p, stream);
    if (best.bn == 128) return launch_glu<128, false, BWD>(p, stream);
    return launch_glu<64, false, BWD>(p, stream);
}

// What both calls ask of their arguments: `a` [M,K] times `b`, scales, the optional outputs,
// and the quantize's (scale, amax, sat); `q` and `t` the codes.
int check_glu(const void* a, const void* b, const float* scale_a, const float* scale_b, int act, const void* h, void* o,
              void* d, const float* scale_q, void* q, void* t, const float* amax, const unsigned long long* sat,
              int64_t M, int64_t F, int64_t K, unsigned flags, const int* status) {
    if (flags & ~static_cast<unsigned>(FP8Q_ACCUMULATE)) return FP8Q_ERR_UNSUPPORTED;
    if (act < FP8Q_ACT_IDENTITY || act > FP8Q_ACT_GELU) return FP8Q_ERR_UNSUPPORTED;
    if (M < 0 || F < 16 || K < 16 || F % 16 != 0 || K % 16 != 0) return FP8Q_ERR_SHAPE;
    const int64_t most = (int64_t(1) << 31) - 2 * BM;
    if (M > most || 2 * F > most || K > most) return FP8Q_ERR_SHAPE;
    if (!b || !scale_a || !scale_b) return FP8Q_ERR_NULL;
    if (M != 0 && !a) return FP8Q_ERR_NULL;
    if ((q || t || sat) && !scale_q) return FP8Q_ERR_NULL;
    if (t && M % 16 != 0) return FP8Q_ERR_SHAPE;
    const void* tensors[] = {a, b, h, o, d, q, t};
    for (const void* x : tensors)
        if (!aligned16(x)) return FP8Q_ERR_ALIGN;
    if (!aligned_to(scale_a, 4) || !aligned_to(scale_b, 4) || !aligned_to(scale_q, 4) || !aligned_to(amax, 4) ||
        !aligned_to(sat, 8) || !aligned_to(status, 4))
        return FP8Q_ERR_ALIGN;
    if (!device_is_sm103()) return FP8Q_ERR_UNSUPPORTED;
    return FP8Q_OK;
}

int run_glu(bool bwd, GluArgs p, unsigned flags, cudaStream_t stream) {
    if (!(flags & FP8Q_ACCUMULATE) && (p.amax || p.sat)) {
        if (launch_pdl(clear_quant_kernel, dim3(1), dim3(1), 0, stream, p.amax, p.sat) != cudaSuccess) {
            (void)cudaGetLastError();
            return FP8Q_ERR_CUDA;
        }
    }
    if (p.M == 0) return FP8Q_OK;
    // (a row of h, o or d is a multiple of 32 bytes long, one of q only where F is)
    p.hold = gemm_loads_held();
    p.wide_bf = aligned_to(p.h, 32) && aligned_to(p.o, 32) && aligned_to(p.d, 32);
    p.wide_q = aligned_to(p.q, 32) && p.F % 32 == 0;
    return bwd ? dispatch_glu<true>(p, stream) : dispatch_glu<false>(p, stream);
}

}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" int fp8q_glu_set_tile(int pair, int bn) {
    if (pair == -1) {
        g_glu_tile.store(-1);
        return FP8Q_OK;
    }
    if ((pair != 0 && pair != 1) || (bn != 128 && bn != 192 && bn != 256 && (bn != 64 || pair))) return FP8Q_ERR_UNSUPPORTED;
    g_glu_tile.store((pair << 16) | bn);
    return FP8Q_OK;
}

extern "C" int fp8_glu_fwd(const fp8q_glu_args* args, cudaStream_t stream) {
    if (!args) return FP8Q_ERR_NULL;
    const fp8q_glu_args& a = *args;
    const int st = check_glu(a.x_q, a.w1t_q, a.scale_x, a.scale_w, a.act, nullptr, a.h_out, a.act_out, a.scale_a, a.a_q,
                             a.a_q_t, a.amax_out, a.sat_count, a.M, a.F, a.K, a.flags, a.status);
    if (st != FP8Q_OK && st != FP8Q_ERR_UNSUPPORTED) return st;
    if (a.M != 0 && !a.act_out && !a.a_q && !a.a_q_t) return FP8Q_ERR_NULL;
    if (st != FP8Q_OK) return st;
    GluArgs p = {};
    p.x = a.x_q;
    p.w = a.w1t_q;
    p.o = static_cast<uint16_t*>(a.h_out);
    p.d = static_cast<uint16_t*>(a.act_out);
    p.q = static_cast<uint8_t*>(a.a_q);
    p.t = static_cast<uint8_t*>(a.a_q_t);
    p.scale_a = a.scale_x;
    p.scale_b = a.scale_w;
    p.scale_q = a.scale_a;
    p.amax = a.amax_out;
    p.sat = a.sat_count;
    p.status = a.status;
    p.M = a.M;
    p.F = a.F;
    p.K = a.K;
    p.act = a.act;
    return run_glu(false, p, a.flags, stream);
}

extern "C" int fp8_gemm_dgrad_glu(const fp8q_dgrad_glu_args* args, cudaStream_t stream) {
    if (!args) return FP8Q_ERR_NULL;
    const fp8q_dgrad_glu_args& a = *args;
    const int st = check_glu(a.dy_q, a.w2_q, a.scale_dy, a.scale_w, a.act, a.h, a.dh, nullptr, a.scale_dh, a.dh_q,
                             a.dh_q_t, a.amax_out, a.sat_count, a.M, a.F, a.N, a.flags, a.status);
    if (st != FP8Q_OK && st != FP8Q_ERR_UNSUPPORTED) return st;
    if (a.M != 0 && (!a.h || (!a.dh && !a.dh_q && !a.dh_q_t))) return FP8Q_ERR_NULL;
    if (st != FP8Q_OK) return st;
    GluArgs p = {};
    p.x = a.dy_q;
    p.w = a.w2_q;
    p.h = static_cast<const uint16_t*>(a.h);
    p.o = static_cast<uint16_t*>(a.dh);
    p.q = static_cast<uint8_t*>(a.dh_q);
    p.t = static_cast<uint8_t*>(a.dh_q_t);
    p.scale_a = a.scale_dy;
    p.scale_b = a.scale_w;
    p.scale_q = a.scale_dh;
    p.amax = a.amax_out;
    p.sat = a.sat_count;
    p.status = a.status;
    p.M = a.M;
    p.F = a.F;
    p.K = a.N;
    p.act = a.act;
    return run_glu(true, p, a.flags, stream);
}
