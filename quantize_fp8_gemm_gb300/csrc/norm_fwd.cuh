// norm_fwd.cuh -- the one-pass kernels of layer_norm_fwd, which norm_fwd.cu
// launches; each element type is a translation unit of its own (norm_fwd_*.cu),
// so that they compile side by side.
#pragma once

#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>

namespace fp8q {

template <typename T>
struct FwdParams {
    int64_t M, N;
    const T* x;
    int64_t ldx;
    const T* res;
    int64_t ld_res;
    T* r_out;
    int64_t ld_r;
    Params<T> w, b;
    float eps;
    T* y;
    int64_t ldy;
    float* mean;
    float* rstd;
    Dropout drop;
    QuantOut quant;
};

namespace {

// One pass over rows of 16-byte pieces.  One wave of CTAs takes rows in turn;
// the next rows' pieces are in flight in a ring of S rows in shared memory, and
// the row at hand is in registers from its one read to its one write.
//   NARROW  `team` lanes (a power of two <= 32) of a warp take a row, up to 64
//           columns a lane; statistics by shuffles
//   WIDE    a CTA of up to 256 threads takes a row, 32 columns a thread
//   BROAD   the same with up to 512 threads, whose registers hold no weights
// A CTA's warps each form the mean and the squared deviations of their part; the
// parts are joined in one exchange:  mean = sum n_w mean_w / N,
// sum dev^2 = sum (dev^2_w + n_w (mean_w - mean)^2).
// SHIFT: rows off the 16-byte grid (norm_ops.cuh).  A thread copies its own
// granule, the last lane of a team one more; a lane reads its own and the next.
// Without SHIFT a thread reads what it copied, and waits for its own copies only.
//
// What bounds it: memory from about 1000 columns and 10^4 rows on, as the ring
// keeps 40 KB or more of loads in flight a multiprocessor whatever the registers
// hold.  A warp a row costs the fewest instructions (statistics are ten shuffles a
// row, weights stay in registers); a CTA a row pays a barrier.  Packed float32
// pairs (f32x2) halve the arithmetic.  With dropout it is memory and latency together:
// a piece of eight columns takes about 235 instructions, 70 of them the generator's, in
// 168 registers, and the 11 warps of a multiprocessor issue in 52 % of the cycles
// (32768 x 1600 with codes: multiply pipe 53 %, memory 62 % of its peak).
// Measured on GB300 (share of the measured copy rate, 6785 GB/s): bf16 131072 x
// 1600 148 us (0.83), with residual 273 us (0.91), with dropout, residual and
// E4M3 codes 309 us (0.90); 32768 x 4096 84 us (0.95); 8192 x 16384 109 us (0.72);
// 131072 x 128 16.6 us (0.60: two rows a warp, instruction-bound); off the grid
// float32 65536 x 1001 92 us (0.84), bf16 16384 x 1001 21 us (0.46: cutting and
// joining the granules makes 8 instructions an element 26, which 11 warps issue in
// 46 % of the cycles, the memory at 18 % of its peak).  The register-only form before
// the ring (loads in registers, weights from L1) took 272 us at 131072 x 1600.
enum FwdMode { NARROW, WIDE, BROAD };

// With 40 columns a lane or more the generator's registers beside 128 of weights
// would leave two warps a scheduler: the CTA's weights are then in shared memory
// (131072 x 1600 with dropout: 429 us with them from L1, 317 from shared memory;
// at 24 columns registers are better, 65536 x 768 66 against 72 us), as BROAD's
// are where one input's ring leaves room for them (8192 x 16384: 151 us with the
// weights from L2, twice the row's own bytes in every row, 107 from shared memory).
__host__ __device__ constexpr bool weights_held(int columns, bool drop, FwdMode mode) {
    return mode != BROAD && !(drop && columns >= 40);
}
__host__ __device__ constexpr bool weights_shared(int columns, bool drop, bool res, FwdMode mode) {
    return !weights_held(columns, drop, mode) && (mode == NARROW || (mode == BROAD && !res));
}
// Rows of the ring: what leaves room for three CTAs a multiprocessor (131072 x 1600
// with dropout and residual: 308 us with two rows, 372 with three and two CTAs), or
// fits at all.
__host__ __device__ constexpr int ring_rows(int C, int columns, bool drop, bool res, FwdMode mode) {
    if (mode == BROAD) return C == 8 ? 1 : 2;
    return drop && res && columns >= 40 ? 2 : 3;
}

template <typename T, int C, bool DROP, bool RES, FwdMode MODE, bool SHIFT>
__global__ void __launch_bounds__(MODE == BROAD ? 512 : MODE == WIDE ? 256 : 128,
                                  MODE == NARROW && DROP && C * 16 / sizeof(T) >= 32 ? 3 : 1)
ln_fwd_ring_kernel(const FwdParams<T> p, int team) {
    extern __shared__ uint4 s_ring[];  // [stage][x, residual][c][slot]
    __shared__ float4 s_warp[2][16];   // a warp's n, n * mean, mean, squared deviations
    constexpr int V = 16 / sizeof(T), H = V / 2, TENSORS = RES ? 2 : 1;
    constexpr int S = ring_rows(C, C * V, DROP, RES, MODE);
    constexpr bool kHeld = weights_held(C * V, DROP, MODE), kCta = MODE != NARROW;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if constexpr (C > 1 || kCta) team = 32;
    // piece c of this thread is piece t + 32 c of its row: a warp's are adjacent
    const int t = kCta ? warp * 32 * C + lane : lane & (team - 1);
    const int N = static_cast<int>(p.N), pieces = SHIFT ? (N + V - 1) / V : N / V;
    const float inv_n = 1.0f / static_cast<float>(N);
    const f32x2 zero2 = pair_of(0.0f, 0.0f);
    // whether this thread's piece c lies in the row: all but the last of a warp's do
    auto has = [&](int c) { return (!kCta && c < C - 1) || t + c * 32 < pieces; };
    uint4 carry = make_uint4(0, 0, 0, 0);
    auto count = [&](int c) { return SHIFT && (kCta || c == C - 1) ? min(V, N - (t + c * 32) * V) : V; };  // of its elements, where it does
    // (SHIFT) store of piece c; a row's first piece is in its first lane's first, its last one in the last
    auto put = [&](uint4 q, uint4& carried, T* start, int c, int valid) {
        const bool head = c == 0 && (kCta ? lane : t) == 0, tail = t + c * 32 == pieces - 1 || (kCta && c == C - 1 && lane == 31);
        if (C == 1 || (kCta && c == 0)) store_shifted<T, true, true>(q, carried, start, t + c * 32, valid, head, tail);
        else if (c == 0) store_shifted<T, true, false>(q, carried, start, t + c * 32, valid, head, tail);
        else if (c == C - 1 || kCta) store_shifted<T, false, true>(q, carried, start, t + c * 32, valid, head, tail);
        else store_shifted<T, false, false>(q, carried, start, t + c * 32, valid, head, tail);
    };
    pdl_wait();

    // [warp of a CTA's row][w, b][four columns of a piece][c][lane]: lanes 16 bytes apart
    constexpr bool kShared = weights_shared(C * V, DROP, RES, MODE);
    float4* const s_par = reinterpret_cast<float4*>(s_ring + nw * (S * TENSORS * C * warp_slots(SHIFT, !kCta && C == 1))) +
                          (kCta ? warp * (2 * (V / 4) * C * 32) : 0) + lane;
    f32x2 w[kHeld ? C : 1][H], b[kHeld ? C : 1][H];
    int own = 0;  // elements of this thread; of this warp later
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < H; ++i) w[c][i] = b[c][i] = zero2;
        }
        if (!has(c)) continue;
        own += count(c);
        if constexpr (kHeld) {
            load_params2<T, V, SHIFT>(p.w, (t + c * 32) * V, N, w[c]);
            load_params2<T, V, SHIFT>(p.b, (t + c * 32) * V, N, b[c]);
        }
        if constexpr (kShared) {
            if (kCta || warp == c % 4) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    f32x2 f[H];
                    load_params2<T, V, SHIFT>(q ? p.b : p.w, (t + c * 32) * V, N, f);
#pragma unroll
                    for (int i = 0; i < V / 4; ++i) {
                        const float2 x = split(f[2 * i]), y = split(f[2 * i + 1]);
                        s_par[((q * (V / 4) + i) * C + c) * 32] = make_float4(x.x, x.y, y.x, y.y);
                    }
                }
            }
        }
    }
    if constexpr (kShared) __syncthreads();
    float inv_own = inv_n;  // 1 / (elements whose mean a warp forms)
    if constexpr (kCta) {
        own = __reduce_add_sync(0xFFFFFFFFu, own);
        inv_own = own ? 1.0f / static_cast<float>(own) : 0.0f;
        if (threadIdx.x < 32) s_warp[threadIdx.x >> 4][threadIdx.x & 15] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncthreads();
    }
    Philox g;
    if constexpr (DROP) g = Philox(p.drop.rng);
    const uint64_t first_m0 = kPhiloxM0 * static_cast<uint32_t>(t * (V / 4));  // of this thread's first piece
    const float s = p.quant.on ? *p.quant.scale : 0.0f;
    uint32_t amax = 0, amax2 = 0, nsat = 0;

    const int rows_warp = kCta ? 1 : 32 / team, rows_cta = kCta ? 1 : rows_warp * nw;
    // (M is below 2^31, and so few rows ahead of it below 2^32)
    const uint32_t M = static_cast<uint32_t>(p.M), stride = gridDim.x * rows_cta, base0 = blockIdx.x * rows_cta;
    const uint32_t sub = kCta ? 0 : warp * rows_warp + lane / team;
    constexpr bool kRun = C <= 2;
    RowWalk<const T, kRun> x_in(p.x, p.ldx, base0 + sub, stride), res_in(p.res, p.ld_res, base0 + sub, stride);
    RowWalk<const T, kRun> x_at = x_in, res_at = res_in;
    RowWalk<T, kRun> r_at(p.r_out, p.ld_r, base0 + sub, stride), y_at(p.y, p.ldy, base0 + sub, stride);
    RowWalk<uint8_t, kRun> q_at(p.quant.q, p.N, base0 + sub, stride);
    constexpr int kSlots = warp_slots(SHIFT, !kCta && C == 1), kStage = TENSORS * C * kSlots;
    uint4* const ring = s_ring + warp * (S * kStage) + lane + (SHIFT ? lane / team : 0);  // [stage][tensor][c][slot]
    const bool team_end = SHIFT && (kCta ? lane == 31 : t == team - 1);
    const uint32_t ring_at = smem_u32(ring);
    auto fill_tensor = [&](uint32_t to, const T* start) {
        const uint32_t mis = SHIFT ? granule_offset(start) : 0;
        const uint8_t* first = reinterpret_cast<const uint8_t*>(start) - mis;
        const int end = N * static_cast<int>(sizeof(T)) + static_cast<int>(mis);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (SHIFT) {
                if (!kCta && c < C - 1) copy_granules<true>(to + c * kSlots * 16, first, t + c * 32, end, team_end);
                else copy_granules<false>(to + c * kSlots * 16, first, t + c * 32, end, team_end);
            } else if (has(c)) {
                cp_async16(to + c * kSlots * 16, start + t * V + c * 32 * V);
            }
        }
    };
    // the pieces of a row; nothing for a row past the last, whose results are not used
    auto fill = [&](int stage, uint32_t row) {
        if (row < M) {
            const uint32_t to = ring_at + stage * kStage * 16;
            fill_tensor(to, x_in.at(row));
            if constexpr (RES) fill_tensor(to + C * kSlots * 16, res_in.at(row));
        }
        cp_async_commit();
        x_in.next();
        if constexpr (RES) res_in.next();
    };
    if constexpr (!SHIFT) {  // pieces past the row are zeros in every stage, and stay so
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (!has(c))
                for (int k = 0; k < S * TENSORS; ++k) ring[(k * C + c) * kSlots] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);

    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
    int stage = 0, buf = 0;
    // where a warp takes one row, it is done at its own last; where it shares a barrier or
    // its lanes take several, at the CTA's
    constexpr bool kOwnEnd = MODE == NARROW && C > 1;
    for (uint32_t base = base0; (kOwnEnd ? base + sub : base) < M; base += stride) {
        const uint32_t row = base + sub;
        const bool in = kOwnEnd || kCta || row < M;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        cp_async_wait<S - 1>();
        const uint4* at = ring + stage * kStage;
        if constexpr (SHIFT) __syncwarp();
        uint64_t row_m0 = 0;
        if constexpr (DROP) row_m0 = g.row(row);
        const uint32_t mis_x = SHIFT ? granule_offset(x_at.at(row)) : 0;
        const uint32_t mis_r = SHIFT && RES ? granule_offset(res_at.at(row)) : 0;
        T* r_row = r_at.at(row);
        f32x2 v[C][H], sum2 = zero2;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Piece<T, V> a;
            a.raw = read_piece<T, SHIFT>(at + c * kSlots, mis_x);
            if constexpr (DROP || RES) {
                unpack2(a, v[c]);
                if constexpr (DROP) {
                    uint32_t words[V];
                    words_at<V>(g, first_m0 + kPhiloxM0 * static_cast<uint32_t>(c * 32 * (V / 4)), row_m0, words);
#pragma unroll
                    for (int i = 0; i < H; ++i) v[c][i] = dropped2(mul2(v[c][i], inv2), words[2 * i], words[2 * i + 1], p.drop);
                }
                if constexpr (RES) {
                    Piece<T, V> r;
                    r.raw = read_piece<T, SHIFT>(at + (C + c) * kSlots, mis_r);
                    f32x2 f[H];
                    unpack2(r, f);
#pragma unroll
                    for (int i = 0; i < H; ++i) v[c][i] = add2(f[i], v[c][i]);
                }
                pack2(a, v[c]);
            }
            if (p.r_out) {
                if constexpr (SHIFT) put(a.raw, carry, r_row, c, in && has(c) ? count(c) : 0);
                else if (in && has(c)) a.store(r_row + t * V + c * 32 * V);
            }
            unpack2(a, v[c]);
            if constexpr (SHIFT) {
                if (t + c * 32 >= pieces || count(c) < V) zero_from<V>(v[c], t + c * 32 < pieces ? count(c) : 0);
            }
            f32x2 part = add2(v[c][0], v[c][1]);
            if constexpr (H == 4) part = add2(part, add2(v[c][2], v[c][3]));
            sum2 = add2(sum2, part);
        }
        const float2 halves = split(sum2);
        float sum = halves.x + halves.y;
        sum = team_sum<C == 1 && !kCta>(sum, team);
        float mean = sum * inv_own;
        f32x2 shift = pair_of(-mean, -mean), dev2[2] = {zero2, zero2};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!has(c)) continue;
            f32x2 d[H];
#pragma unroll
            for (int i = 0; i < H; ++i) d[i] = add2(v[c][i], shift);
            if (SHIFT && count(c) < V) zero_from<V>(d, count(c));
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if constexpr (!kCta) v[c][i] = d[i];
                dev2[i & 1] = fma2(d[i], d[i], dev2[i & 1]);
            }
        }
        const float2 devs = split(add2(dev2[0], dev2[1]));
        float dev = devs.x + devs.y;
        dev = team_sum<C == 1 && !kCta>(dev, team);
        if constexpr (kCta) {
            // two buffers: a warp that runs ahead writes the other one, and cannot reach this one
            // again before every warp has passed the next row's barrier
            const float n = static_cast<float>(own);
            if (lane == 0) s_warp[buf][warp] = make_float4(n, n * mean, mean, dev);
            __syncthreads();
            constexpr int kWarps = MODE == WIDE ? 8 : 16;  // absent ones are zeros
            sum = dev = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) sum += s_warp[buf][k].y;
            mean = sum * inv_n;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 f = s_warp[buf][k];
                const float m = f.z - mean;
                dev += __fmaf_rn(f.x * m, m, f.w);
            }
            buf ^= 1;
            shift = pair_of(-mean, -mean);
        }
        const float rstd = 1.0f / sqrtf(__fmaf_rn(dev, inv_n, p.eps));
        const f32x2 scale = pair_of(rstd, rstd);
        T* y_row = y_at.at(row);
        uint8_t* q_row = q_at.at(row);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int valid = in && has(c) ? count(c) : 0;
            if (!SHIFT && valid == 0) continue;
            f32x2 wl[H], bl[H];
            if constexpr (!kHeld) {
                if constexpr (kShared) {
#pragma unroll
                    for (int i = 0; i < V / 4; ++i) {
                        const float4 fw = s_par[(i * C + c) * 32], fb = s_par[((V / 4 + i) * C + c) * 32];
                        wl[2 * i] = pair_of(fw.x, fw.y);
                        wl[2 * i + 1] = pair_of(fw.z, fw.w);
                        bl[2 * i] = pair_of(fb.x, fb.y);
                        bl[2 * i + 1] = pair_of(fb.z, fb.w);
                    }
                } else if (valid > 0) {
                    load_params2<T, V, SHIFT>(p.w, (t + c * 32) * V, N, wl);
                    load_params2<T, V, SHIFT>(p.b, (t + c * 32) * V, N, bl);
                }
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const f32x2 d = kCta ? add2(v[c][i], shift) : v[c][i];
                v[c][i] = fma2(mul2(d, scale), kHeld ? w[kHeld ? c : 0][i] : wl[i], kHeld ? b[kHeld ? c : 0][i] : bl[i]);
            }
            Piece<T, V> y;
            pack2(y, v[c]);
            if (p.y) {
                if constexpr (SHIFT) put(y.raw, carry, y_row, c, valid);
                else y.store(y_row + t * V + c * 32 * V);
            }
            if (p.quant.on && valid > 0) {
                uint8_t* dst = p.quant.q ? q_row + t * V + c * 32 * V : nullptr;
                const bool whole = !SHIFT || (valid == V && (reinterpret_cast<uintptr_t>(dst) & (V - 1)) == 0);
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    if (whole) {
                        if (p.quant.fmt == FP8Q_E5M2) quant_bf16x8<FP8Q_E5M2>(s, y.raw, dst, amax2, nsat);
                        else quant_bf16x8<FP8Q_E4M3>(s, y.raw, dst, amax2, nsat);
                        continue;
                    }
                }
                quant_piece<T, V>(p.quant, s, y, dst, valid, whole, amax, nsat);
            }
        }
        if (in && t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        x_at.next();
        res_at.next();
        r_at.next();
        y_at.next();
        q_at.next();
        if constexpr (SHIFT) __syncwarp();  // the granules that a neighbour read may be overwritten now
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
    if (p.quant.on) publish_quant(p.quant, max(amax, max16x2(amax2) << 16), nsat);
}

template <typename T, int C, bool DROP, bool RES, FwdMode MODE, bool SHIFT>
cudaError_t launch_ring_as(const FwdParams<T>& p, int team, unsigned block, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    // one wave: as many CTAs as run at a time (kept by device and CTA size)
    static DeviceTable<17> table;
    const auto kern = ln_fwd_ring_kernel<T, C, DROP, RES, MODE, SHIFT>;
    size_t smem = size_t(ring_rows(C, C * V, DROP, RES, MODE)) * (RES ? 2 : 1) * C * (block / 32) *
                        warp_slots(SHIFT, MODE == NARROW && C == 1) * 16;
    if (weights_shared(C * V, DROP, RES, MODE)) smem += size_t(2) * C * 32 * V * sizeof(float) * (MODE == NARROW ? 1 : block / 32);
    int n = 0;
    const cudaError_t e = resident_ctas(table, kern, block, smem, kMaxRing, &n);
    if (e != cudaSuccess) return e;
    const int64_t rows = MODE == NARROW ? 128 / team : 1;
    const int64_t grid = std::min<int64_t>((p.M + rows - 1) / rows, int64_t(n) * sm_count());
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, p, team);
}

template <typename T, int C, FwdMode MODE, bool SHIFT>
cudaError_t launch_ring(const FwdParams<T>& p, int team, unsigned block, cudaStream_t stream) {
    if (p.drop.on)
        return p.res ? launch_ring_as<T, C, true, true, MODE, SHIFT>(p, team, block, stream)
                     : launch_ring_as<T, C, true, false, MODE, SHIFT>(p, team, block, stream);
    return p.res ? launch_ring_as<T, C, false, true, MODE, SHIFT>(p, team, block, stream)
                 : launch_ring_as<T, C, false, false, MODE, SHIFT>(p, team, block, stream);
}

}  // namespace

// The one-pass kernels, where the row fits one; cudaErrorNotSupported where it does not.
template <typename T, bool SHIFT>
cudaError_t launch_fwd_ring(const FwdParams<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), kMost = 32 / V;
    const int64_t pieces = (p.N + V - 1) / V;
    const int team = team_of(pieces);
    switch ((pieces + team - 1) / team) {
        case 1: return launch_ring<T, 1, NARROW, SHIFT>(p, team, 128, stream);
        case 2: return launch_ring<T, 2, NARROW, SHIFT>(p, team, 128, stream);
        case 3: return launch_ring<T, 3, NARROW, SHIFT>(p, team, 128, stream);
        case 4: return launch_ring<T, 4, NARROW, SHIFT>(p, team, 128, stream);
        case 5: return launch_ring<T, 5, NARROW, SHIFT>(p, team, 128, stream);
        case 6: return launch_ring<T, 6, NARROW, SHIFT>(p, team, 128, stream);
        case 7: return launch_ring<T, 7, NARROW, SHIFT>(p, team, 128, stream);
        case 8: return launch_ring<T, 8, NARROW, SHIFT>(p, team, 128, stream);
        default: break;
    }
    if (pieces <= 256 * kMost) {
        const int64_t warps = (pieces + 32 * kMost - 1) / (32 * kMost);
        const unsigned block = static_cast<unsigned>(warps) * 32;
        const int64_t c = (pieces + 32 * warps - 1) / (32 * warps);  // kMost, or less with few warps
        if constexpr (V == 8) {
            if (c <= 3) return launch_ring<T, 3, WIDE, SHIFT>(p, 32, block, stream);
        } else {
            if (c <= 5) return launch_ring<T, 5, WIDE, SHIFT>(p, 32, block, stream);
            if (c == 6) return launch_ring<T, 6, WIDE, SHIFT>(p, 32, block, stream);
            if (c == 7) return launch_ring<T, 7, WIDE, SHIFT>(p, 32, block, stream);
        }
        return launch_ring<T, kMost, WIDE, SHIFT>(p, 32, block, stream);
    }
    if (pieces <= 512 * kMost) return launch_ring<T, kMost, BROAD, SHIFT>(p, 32, threads_of(pieces, kMost), stream);
    return cudaErrorNotSupported;
}

}  // namespace fp8q
