// glu.cu -- the gated feed-forward block's kernels: both projections, the activation,
// the product and its quantize in one GEMM (fp8_glu_fwd), and the gradient of that in
// the down-projection's dgrad (fp8_gemm_dgrad_glu).
//
//   forward   [g | u] = X W1 (E4M3 x E4M3, FP32 sums); a = act(g) u; q = E4M3(BF16(a) s)
//   backward  dA = dY W2^T (E5M2 x E4M3, FP32 sums); dg = dA u act'(g), du = dA act(g)
//
// Both are the tcgen05 GEMM D[M, .] = A[M,K] . B[., K]^T of gemm_parts.cuh's pieces with
// an epilogue of their own.  A CTA is 10 warps, persistent over output tiles:
//   warp 0     TMA producer: k-blocks of 128 bytes a row into a ring of stages
//   warp 1     MMA issuer: kind::f8f6f4 into one of two TMEM accumulators
//   warps 2-9  epilogue: two warps a TMEM lane quarter, alternate 32-column chunks
// PAIR: a cluster of two CTAs, 256 rows a tile, cta_group::2.
//
// The forward tile of BN accumulator columns is BN / 2 columns of the gate and the same
// BN / 2 of the up-projection side by side, so that a thread holds g and u of one element
// and nothing but the product leaves the SM.  In a pair each CTA loads one of the two as
// its half of B: the MMA reads B's first half from the leader's shared memory (the gate's
// rows of W1^T) and its second from the peer's (the up-projection's).
//
// The backward tile is BN columns of dA; the chunks of g and u that it needs come by TMA
// into two buffers a warp, asked for one chunk ahead (the first before the accumulator is
// ready), and the gradients are written over them.
//
// Every wait is bounded as in gemm.cu: on time-out the CTA sets FP8Q_DEV_TIMEOUT, lets its
// copies and MMAs land (bounded), frees TMEM and exits.
#include "common.cuh"
#include "gemm_parts.cuh"
#include "glu_ops.cuh"
#include "norm_ops.cuh"
#include "quant_ops.cuh"

#include <algorithm>

namespace fp8q {

namespace {

constexpr int kGluWarps = 8;                      // epilogue warps
constexpr int kGluThreads = 64 + 32 * kGluWarps;
constexpr int kBox = 32 * 32;                     // elements of a box: 32 rows x 32 columns

// Tensor maps of a call; one that a call has no tensor for is a copy of `a`, never used.
// h (read), o (h_out or dh), q, t: the halves (gate, up) of a [M,2F] or [2F,M] tensor, each
// a tensor of its own width, so that a box at a half's ragged end is clipped there.
struct GluMaps {
    CUtensorMap a, b, h0, h1, o0, o1, d, q0, q1, t0, t1;
};

struct GluArgs {
    const float* scale_a;
    const float* scale_b;
    const float* scale_q;
    float* amax;
    unsigned long long* sat;
    int* status;
    int64_t M, F, K;
    uint32_t idesc;
    int act;
    bool has_o, has_d, has_q, has_t;  // h_out or dh; act_out; codes; transposed codes
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
    // forward: g, u and a (BF16 boxes), codes and their transpose; backward: two buffers of
    // g and u, and both halves' codes and transposes
    static constexpr int WARP_BYTES = BWD ? 2 * 4 * kBox + 4 * kBox : 6 * kBox + 2 * kBox;
    static constexpr int BAR_BYTES = 512;
    static constexpr int RING = 232448 - 512 - BAR_BYTES - 1024 - kGluWarps * WARP_BYTES;
    static constexpr int STAGES = RING / STAGE_BYTES < 8 ? RING / STAGE_BYTES : 8;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + kGluWarps * WARP_BYTES + BAR_BYTES + 1024;
    static constexpr int TMEM_COLS = 2 * BN <= 64 ? 64 : 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
    static constexpr int TILE_M = PAIR ? 2 * BM : BM;
    static constexpr int CHUNKS = OUT / 32;
    static_assert(OUT % 32 == 0 && BN <= 256 && STAGES >= 2 && (B_ROWS * BK) % 1024 == 0, "tile shape");
    static_assert((2 * STAGES + 2 * ACCS + 1 + 2 * kGluWarps) * 8 + 16 <= BAR_BYTES, "barrier area");
};

// The codes of one chunk (32 columns of this lane's row, packed BF16) into `codes` (32 x 32
// bytes, lane r's row at 32 r) and, transposed, into `turned` (column j at 32 j).  Four lanes
// turn 4 x 4 bytes by two exchanges: first neighbouring lanes swap odd for even bytes, then
// pairs of lanes high for low halves; lane 4 k + i then holds rows 4 k .. 4 k + 3 of column
// 4 w + i, and a warp's stores of a word fill all banks.  (A byte store a code and the shifts
// before it, 56 instructions for 32 codes against 40.)
template <int FMT>
__device__ __forceinline__ void glu_codes(const uint32_t (&v)[16], float s, uint8_t* codes, uint8_t* turned, int lane,
                                          bool want_codes, bool want_turned, uint32_t& amax2, uint32_t& nsat) {
    uint32_t q[8], all = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint4 p = make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        all = __vmaxu2(all, __vmaxu2(__vmaxu2(p.x & 0x7FFF7FFFu, p.y & 0x7FFF7FFFu),
                                     __vmaxu2(p.z & 0x7FFF7FFFu, p.w & 0x7FFF7FFFu)));
        const uint2 c = cast8_codes<FMT>(p, s);
        q[2 * g] = c.x;
        q[2 * g + 1] = c.y;
    }
    amax2 = __vmaxu2(amax2, all);
    if (!(__fmul_rn(__uint_as_float(max16x2(all) << 16), s) <= fp8_max_value(FMT))) {  // (a NaN counts the others too)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            nsat += sat_count8<FMT>(make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]), s);
    }
    if (want_codes) {
        *reinterpret_cast<uint4*>(codes + lane * 32) = make_uint4(q[0], q[1], q[2], q[3]);
        *reinterpret_cast<uint4*>(codes + lane * 32 + 16) = make_uint4(q[4], q[5], q[6], q[7]);
    }
    if (want_turned) {
        const uint32_t sel1 = lane & 1 ? 0x3715u : 0x6240u, sel2 = lane & 2 ? 0x3276u : 0x5410u;
        uint8_t* to = turned + (lane & 3) * 32 + (lane >> 2) * 4;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            uint32_t x = __byte_perm(q[w], __shfl_xor_sync(0xFFFFFFFFu, q[w], 1), sel1);
            x = __byte_perm(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2), sel2);
            *reinterpret_cast<uint32_t*>(to + w * 128) = x;
        }
    }
}

// The magnitudes alone (a call that wants a maximum but no codes).
__device__ __forceinline__ void glu_amax(const uint32_t (&v)[16], uint32_t& amax2) {
#pragma unroll
    for (int j = 0; j < 16; ++j) amax2 = __vmaxu2(amax2, v[j] & 0x7FFF7FFFu);
}

// 32 packed BF16 columns of this lane's row into a 32 x 32 box in the 64-byte swizzle.
__device__ __forceinline__ void put_box(uint8_t* box, int lane, const uint32_t (&v)[16]) {
    const int sw = (lane >> 1) & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ sw) << 4)) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

__device__ __forceinline__ f32x2 acc_pair(uint32_t a, uint32_t b) { return pair_of(__uint_as_float(a), __uint_as_float(b)); }

template <int ACT>
__device__ __forceinline__ void glu_products(const uint32_t (&g)[32], const uint32_t (&u)[32], float inv,
                                             uint32_t (&a)[16]) {
    const f32x2 inv2 = twice(inv);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        a[j] = bf16x2_of(mul2(glu_act<ACT>(mul2(acc_pair(g[2 * j], g[2 * j + 1]), inv2)),
                              mul2(acc_pair(u[2 * j], u[2 * j + 1]), inv2)));
}

// The accumulator's 32 columns of this lane's row as packed BF16.
__device__ __forceinline__ void glu_stored(const uint32_t (&r)[32], float inv, uint32_t (&h)[16]) {
    const f32x2 inv2 = twice(inv);
#pragma unroll
    for (int j = 0; j < 16; ++j) h[j] = bf16x2_of(mul2(acc_pair(r[2 * j], r[2 * j + 1]), inv2));
}

// dA of this lane's row (32 columns), its g and u from the boxes -> packed BF16 dg and du.
template <int ACT>
__device__ __forceinline__ void glu_gradients(const uint32_t (&r)[32], float inv, const uint8_t* gbox,
                                              const uint8_t* ubox, int lane, uint32_t (&dg)[16], uint32_t (&du)[16]) {
    const int sw = (lane >> 1) & 3;
    const f32x2 inv2 = twice(inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int at = lane * 64 + ((k ^ sw) << 4);
        const uint4 g4 = *reinterpret_cast<const uint4*>(gbox + at), u4 = *reinterpret_cast<const uint4*>(ubox + at);
        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 d = mul2(acc_pair(r[8 * k + 2 * j], r[8 * k + 2 * j + 1]), inv2);
            f32x2 f, slope;
            glu_act_grad<ACT>(f32x2_of(gw[j]), f, slope);
            dg[4 * k + j] = bf16x2_of(mul2(mul2(d, f32x2_of(uw[j])), slope));
            du[4 * k + j] = bf16x2_of(mul2(d, f));
        }
    }
}

template <int BN, bool PAIR, bool BWD>
__global__ void __launch_bounds__(kGluThreads, 1)
glu_kernel(const __grid_constant__ GluMaps maps, const GluArgs p) {
    using C = GluCfg<BN, PAIR, BWD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stage0 = smem + C::STAGES * C::STAGE_BYTES;  // the epilogue warps' buffers, 1024-aligned
    uint64_t* bars = reinterpret_cast<uint64_t*>(stage0 + kGluWarps * C::WARP_BYTES);
    uint64_t* full = bars;
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* tempty = tfull + C::ACCS;
    uint64_t* drain = tempty + C::ACCS;
    uint64_t* loaded = drain + 1;  // backward: [warp][buffer]
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(loaded + 2 * kGluWarps);
    volatile int* abort_flag = reinterpret_cast<int*>(tmem_holder) + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int64_t num_n = (p.F + C::OUT - 1) / C::OUT;
    const int64_t num_tiles = ((p.M + C::TILE_M - 1) / C::TILE_M) * num_n;
    const int64_t first_tile = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const int64_t tile_stride = PAIR ? gridDim.x / 2 : gridDim.x;
    const int num_kb = static_cast<int>((p.K + BK - 1) / BK);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < C::ACCS; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), kGluWarps * (PAIR ? 2 : 1));
        }
        mbar_init(smem_u32(drain), 1);
        for (int i = 0; i < 2 * kGluWarps; ++i) mbar_init(smem_u32(&loaded[i]), 1);
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
            for (int64_t tile = first_tile; tile < num_tiles && ok; tile += tile_stride) {
                const int32_t m0 = static_cast<int32_t>((tile / num_n) * C::TILE_M + rank * BM);
                const int32_t n0 = static_cast<int32_t>((tile % num_n) * C::OUT);
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
                        mbar_arrive_expect_tx(fb, C::TX_BYTES);
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
            for (int64_t tile = first_tile; tile < num_tiles && ok; tile += tile_stride) {
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
        const int q = warp & 3;           // TMEM lane quarter of this warp
        const int c0 = (warp - 2) / 4;    // its first chunk; every second one is the other warp's
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : smem_u32(&tempty[0]);
        uint8_t* buf = stage0 + (warp - 2) * C::WARP_BYTES;
        const float inv = 1.0f / (__ldg(p.scale_a) * __ldg(p.scale_b));
        const float s_q = p.scale_q ? __ldg(p.scale_q) : 0.0f;
        uint32_t amax2 = 0, nsat = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true, stored = false;

        auto first_row = [&](int64_t tile) { return (tile / num_n) * C::TILE_M + rank * BM + q * 32; };
        auto first_col = [&](int64_t tile, int c) { return (tile % num_n) * C::OUT + c * 32; };

        // backward: this warp's next chunk of g and u, in the order in which they are used;
        // `asked` of them are on the way or read, `used` of them read
        uint64_t* bar = loaded + 2 * (warp - 2);
        int64_t ask_tile = first_tile;
        int ask_c = c0;
        uint32_t asked = 0, used = 0;
        auto ask = [&]() {
            while (ask_tile < num_tiles && (ask_c >= C::CHUNKS || first_row(ask_tile) >= p.M || first_col(ask_tile, ask_c) >= p.F)) {
                ask_tile += tile_stride;
                ask_c = c0;
            }
            if (ask_tile >= num_tiles) return;
            if (lane == 0) {
                const uint32_t b = smem_u32(&bar[asked & 1]), to = smem_u32(buf + (asked & 1) * 4 * kBox);
                const int32_t x = static_cast<int32_t>(first_col(ask_tile, ask_c)), y = static_cast<int32_t>(first_row(ask_tile));
                mbar_arrive_expect_tx(b, 4 * kBox);
                tma_load_2d(to, &maps.h0, b, x, y);
                tma_load_2d(to + 2 * kBox, &maps.h1, b, x, y);
            }
            ++asked;
            ask_c += 2;
        };
        if constexpr (BWD) ask();

        for (int64_t tile = first_tile; tile < num_tiles; tile += tile_stride) {
            const int64_t row0 = first_row(tile);
            ok = __all_sync(0xFFFFFFFFu, wait_phase(&tfull[acc], acc_phase, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + lane_base + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
            for (int c = c0; c < C::CHUNKS; c += 2) {
                const int64_t col0 = first_col(tile, c);
                if (row0 >= p.M || col0 >= p.F) break;
                const int32_t x = static_cast<int32_t>(col0), y = static_cast<int32_t>(row0);
                if constexpr (!BWD) {
                    uint32_t g[32], u[32], a[16];
                    tmem_ld_2x32_sync(taddr + c * 32, taddr + C::OUT + c * 32, g, u);
                    if (col0 + 32 > p.F) {  // F ends inside the chunk: its last 16 columns are not the gate's
#pragma unroll
                        for (int j = 16; j < 32; ++j) g[j] = u[j] = 0;
                    }
                    switch (p.act) {
                        case FP8Q_ACT_IDENTITY: glu_products<FP8Q_ACT_IDENTITY>(g, u, inv, a); break;
                        case FP8Q_ACT_RELU: glu_products<FP8Q_ACT_RELU>(g, u, inv, a); break;
                        case FP8Q_ACT_RELU2: glu_products<FP8Q_ACT_RELU2>(g, u, inv, a); break;
                        case FP8Q_ACT_SILU: glu_products<FP8Q_ACT_SILU>(g, u, inv, a); break;
                        default: glu_products<FP8Q_ACT_GELU>(g, u, inv, a); break;
                    }
                    if (stored) {  // the last chunk's stores have read the buffers
                        if (lane == 0) bulk_wait_group_read<0>();
                        __syncwarp();
                    }
                    if (p.has_o) {
                        uint32_t hv[16];
                        glu_stored(g, inv, hv);
                        put_box(buf, lane, hv);
                        glu_stored(u, inv, hv);
                        put_box(buf + 2 * kBox, lane, hv);
                    }
                    if (p.has_d) put_box(buf + 4 * kBox, lane, a);
                    if (p.scale_q)
                        glu_codes<FP8Q_E4M3>(a, s_q, buf + 6 * kBox, buf + 7 * kBox, lane, p.has_q, p.has_t, amax2, nsat);
                    else
                        glu_amax(a, amax2);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (p.has_o) {
                            tma_store_2d(&maps.o0, smem_u32(buf), x, y);
                            tma_store_2d(&maps.o1, smem_u32(buf + 2 * kBox), x, y);
                        }
                        if (p.has_d) tma_store_2d(&maps.d, smem_u32(buf + 4 * kBox), x, y);
                        if (p.has_q) tma_store_2d(&maps.q0, smem_u32(buf + 6 * kBox), x, y);
                        if (p.has_t) tma_store_2d(&maps.t0, smem_u32(buf + 7 * kBox), y, x);
                        bulk_commit_group();
                    }
                    stored = true;
                } else {
                    // the stores of the chunk before have read their buffers: the next chunk may be asked for
                    if (stored) {
                        if (lane == 0) bulk_wait_group_read<0>();
                        __syncwarp();
                    }
                    ask();
                    ok = __all_sync(0xFFFFFFFFu, wait_phase(&bar[used & 1], (used >> 1) & 1, abort_flag, p.status));
                    if (!ok) break;
                    uint8_t* box = buf + (used & 1) * 4 * kBox;
                    uint8_t* codes = buf + 8 * kBox;
                    ++used;
                    uint32_t r[32], dg[16], du[16];
                    tmem_ld_x32_sync(taddr + c * 32, r);
                    switch (p.act) {
                        case FP8Q_ACT_IDENTITY: glu_gradients<FP8Q_ACT_IDENTITY>(r, inv, box, box + 2 * kBox, lane, dg, du); break;
                        case FP8Q_ACT_RELU: glu_gradients<FP8Q_ACT_RELU>(r, inv, box, box + 2 * kBox, lane, dg, du); break;
                        case FP8Q_ACT_RELU2: glu_gradients<FP8Q_ACT_RELU2>(r, inv, box, box + 2 * kBox, lane, dg, du); break;
                        case FP8Q_ACT_SILU: glu_gradients<FP8Q_ACT_SILU>(r, inv, box, box + 2 * kBox, lane, dg, du); break;
                        default: glu_gradients<FP8Q_ACT_GELU>(r, inv, box, box + 2 * kBox, lane, dg, du); break;
                    }
                    if (p.has_o) {  // each lane over its own row of g and u
                        put_box(box, lane, dg);
                        put_box(box + 2 * kBox, lane, du);
                    }
                    if (p.scale_q) {
                        glu_codes<FP8Q_E5M2>(dg, s_q, codes, codes + kBox, lane, p.has_q, p.has_t, amax2, nsat);
                        glu_codes<FP8Q_E5M2>(du, s_q, codes + 2 * kBox, codes + 3 * kBox, lane, p.has_q, p.has_t, amax2, nsat);
                    } else {
                        glu_amax(dg, amax2);
                        glu_amax(du, amax2);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (p.has_o) {
                            tma_store_2d(&maps.o0, smem_u32(box), x, y);
                            tma_store_2d(&maps.o1, smem_u32(box + 2 * kBox), x, y);
                        }
                        if (p.has_q) {
                            tma_store_2d(&maps.q0, smem_u32(codes), x, y);
                            tma_store_2d(&maps.q1, smem_u32(codes + 2 * kBox), x, y);
                        }
                        if (p.has_t) {
                            tma_store_2d(&maps.t0, smem_u32(codes + kBox), y, x);
                            tma_store_2d(&maps.t1, smem_u32(codes + 3 * kBox), y, x);
                        }
                        bulk_commit_group();
                    }
                    stored = true;
                }
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster(tempty0 + 8u * acc);
                else mbar_arrive(tempty0 + 8u * acc);
            }
            next_acc<C::ACCS>(acc, acc_phase);
        }
        // no load may still be landing in shared memory when the CTA exits, and every store has read it
        while (BWD && used < asked) {
            wait_phase_drain(&bar[used & 1], (used >> 1) & 1);
            ++used;
        }
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
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
// One of the halves of a tensor that the epilogue moves in 32 x 32 boxes: `rows` rows of
// `cols` elements, `ld` elements apart, BF16 (64-byte swizzle) or bytes (no swizzle).
bool make_box_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, bool bf16) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * (bf16 ? 2 : 1))};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bf16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensors of a call.  Forward: x [M,K], w [2F,K], o = h_out, d = act_out, q [M,F], t [F,M].
// Backward: x = dY [M,K], w = W2 [F,K], h [M,2F], o = dh, q [M,2F], t [2F,M].
struct GluTensors {
    const void* x;
    const void* w;
    const void* h;
    void* o;
    void* d;
    void* q;
    void* t;
};

template <int BN, bool PAIR, bool BWD>
int launch_glu(const GluTensors& io, GluArgs p, cudaStream_t stream) {
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
        cfg.blockDim = dim3(kGluThreads);
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
    const int64_t halves = BWD ? 2 * F : F;  // columns of the codes
    alignas(64) GluMaps maps;
    if (!make_kmajor_map(&maps.a, io.x, M, p.K, BM) || !make_kmajor_map(&maps.b, io.w, BWD ? F : 2 * F, p.K, C::B_BOX))
        return FP8Q_ERR_CUDA;
    maps.h0 = maps.h1 = maps.o0 = maps.o1 = maps.d = maps.q0 = maps.q1 = maps.t0 = maps.t1 = maps.a;
    const auto half = [](const void* base, int64_t bytes) { return static_cast<const uint8_t*>(base) + bytes; };
    bool ok = true;
    if (BWD) ok = make_box_map(&maps.h0, io.h, M, F, 2 * F, true) && make_box_map(&maps.h1, half(io.h, 2 * F), M, F, 2 * F, true);
    if (io.o) ok = ok && make_box_map(&maps.o0, io.o, M, F, 2 * F, true) && make_box_map(&maps.o1, half(io.o, 2 * F), M, F, 2 * F, true);
    if (io.d) ok = ok && make_box_map(&maps.d, io.d, M, F, F, true);
    if (io.q) {
        ok = ok && make_box_map(&maps.q0, io.q, M, F, halves, false);
        if (BWD) ok = ok && make_box_map(&maps.q1, half(io.q, F), M, F, halves, false);
    }
    if (io.t) {
        ok = ok && make_box_map(&maps.t0, io.t, F, M, M, false);
        if (BWD) ok = ok && make_box_map(&maps.t1, half(io.t, F * M), F, M, M, false);
    }
    if (!ok) return FP8Q_ERR_CUDA;
    p.has_o = io.o != nullptr;
    p.has_d = io.d != nullptr;
    p.has_q = io.q != nullptr;
    p.has_t = io.t != nullptr;
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
    cfg.blockDim = dim3(kGluThreads);
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

// The tile, scored as gemm.cu scores its own: waves x a tile's relative time.
template <bool BWD>
int dispatch_glu(const GluTensors& io, const GluArgs& p, cudaStream_t stream) {
    struct Cand { bool pair; int bn; double t; };
    static constexpr Cand kCands[] = {{true, 256, 1.000}, {true, 192, 0.909}, {true, 128, 0.858},
                                      {false, 256, 1.102}, {false, 192, 0.897}, {false, 128, 0.843}, {false, 64, 0.750}};
    const int64_t sms = sm_count();
    Cand best = kCands[5];
    double best_cost = -1.0;
    for (const Cand& c : kCands) {
        if (c.pair && p.M <= BM) continue;
        const int64_t tile_m = c.pair ? 2 * BM : BM, units = c.pair ? sms / 2 : sms, out = BWD ? c.bn : c.bn / 2;
        const int64_t tiles = ((p.M + tile_m - 1) / tile_m) * ((p.F + out - 1) / out);
        const double cost = static_cast<double>((tiles + units - 1) / units) * c.t;
        if (best_cost < 0 || cost < best_cost) { best_cost = cost; best = c; }
    }
    if (best.pair) {
        if (best.bn == 256) return launch_glu<256, true, BWD>(io, p, stream);
        if (best.bn == 192) return launch_glu<192, true, BWD>(io, p, stream);
        return launch_glu<128, true, BWD>(io, p, stream);
    }
    if (best.bn == 256) return launch_glu<256, false, BWD>(io, p, stream);
    if (best.bn == 192) return launch_glu<192, false, BWD>(io, p, stream);
    if (best.bn == 128) return launch_glu<128, false, BWD>(io, p, stream);
    return launch_glu<64, false, BWD>(io, p, stream);
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

int run_glu(bool bwd, const GluTensors& io, const GluArgs& p, unsigned flags, cudaStream_t stream) {
    if (!(flags & FP8Q_ACCUMULATE) && (p.amax || p.sat)) {
        if (launch_pdl(clear_quant_kernel, dim3(1), dim3(1), 0, stream, p.amax, p.sat) != cudaSuccess) {
            (void)cudaGetLastError();
            return FP8Q_ERR_CUDA;
        }
    }
    if (p.M == 0) return FP8Q_OK;
    return bwd ? dispatch_glu<true>(io, p, stream) : dispatch_glu<false>(io, p, stream);
}

}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" int fp8_glu_fwd(const void* x_q, const void* w1t_q, const float* scale_x, const float* scale_w, int act,
                           void* h_out, void* act_out, const float* scale_a, void* a_q, void* a_q_t, float* amax_out,
                           unsigned long long* sat_count, int64_t M, int64_t F, int64_t K, unsigned flags, int* status,
                           cudaStream_t stream) {
    const int st = check_glu(x_q, w1t_q, scale_x, scale_w, act, nullptr, h_out, act_out, scale_a, a_q, a_q_t, amax_out,
                             sat_count, M, F, K, flags, status);
    if (st != FP8Q_OK && st != FP8Q_ERR_UNSUPPORTED) return st;
    if (M != 0 && !act_out && !a_q && !a_q_t) return FP8Q_ERR_NULL;
    if (st != FP8Q_OK) return st;
    GluArgs p = {};
    p.scale_a = scale_x;
    p.scale_b = scale_w;
    p.scale_q = scale_a;
    p.amax = amax_out;
    p.sat = sat_count;
    p.status = status;
    p.M = M;
    p.F = F;
    p.K = K;
    p.act = act;
    return run_glu(false, GluTensors{x_q, w1t_q, nullptr, h_out, act_out, a_q, a_q_t}, p, flags, stream);
}

extern "C" int fp8_gemm_dgrad_glu(const void* dy_q, const void* w2_q, const float* scale_dy, const float* scale_w,
                                  const void* h, int act, void* dh, const float* scale_dh, void* dh_q, void* dh_q_t,
                                  float* amax_out, unsigned long long* sat_count, int64_t M, int64_t N, int64_t F,
                                  unsigned flags, int* status, cudaStream_t stream) {
    const int st = check_glu(dy_q, w2_q, scale_dy, scale_w, act, h, dh, nullptr, scale_dh, dh_q, dh_q_t, amax_out,
                             sat_count, M, F, N, flags, status);
    if (st != FP8Q_OK && st != FP8Q_ERR_UNSUPPORTED) return st;
    if (M != 0 && (!h || (!dh && !dh_q && !dh_q_t))) return FP8Q_ERR_NULL;
    if (st != FP8Q_OK) return st;
    GluArgs p = {};
    p.scale_a = scale_dy;
    p.scale_b = scale_w;
    p.scale_q = scale_dh;
    p.amax = amax_out;
    p.sat = sat_count;
    p.status = status;
    p.M = M;
    p.F = F;
    p.K = N;
    p.act = act;
    return run_glu(true, GluTensors{dy_q, w2_q, h, dh, nullptr, dh_q, dh_q_t}, p, flags, stream);
}
