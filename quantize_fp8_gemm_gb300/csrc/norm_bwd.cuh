// norm_bwd.cuh -- the one-pass kernels of layer_norm_bwd, which norm_bwd.cu
// launches; each element type is a translation unit of its own (norm_bwd_*.cu),
// so that they compile side by side.
#pragma once

#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>

namespace fp8q {

template <typename T>
struct BwdParams {
    int64_t M, N;
    const T* dy;
    int64_t ld_dy;
    const T* r;
    int64_t ld_r;
    const float* mean;
    const float* rstd;
    Params<T> w;
    const T* dres;
    int64_t ld_dres;
    T* dx;
    int64_t ld_dx;
    T* dbranch;
    int64_t ld_db;
    Dropout drop;
    float* part;  // [parts][2][N]: dweight and dbias sums of a set of rows; NULL: not wanted
    int parts;
    float* dweight;  // the results, for a call of one part
    float* dbias;
    bool accumulate;
};

namespace {

// One pass: every input is read once.  A thread keeps its C pieces' columns for
// all the rows that its CTA takes (row blockIdx.x, + the grid, ...), so the
// column sums stay in registers until the end.  The next rows' pieces are in
// flight in a ring of S rows in shared memory, filled by cp.async: a thread
// copies and reads its own pieces only, so it waits for its own copies and no
// barrier guards the ring.  SHIFT: rows off the 16-byte grid (norm_ops.cuh); a
// lane then reads its own granule and the next lane's.
//   NARROW  `team` lanes (a power of two <= 32) of a warp take a row, up to four
//           pieces a lane: the row's two sums are shuffles
//   WIDE    `team` warps take a row, three or four pieces a lane, and exchange
//           their sums at a barrier of their own; a CTA is several such groups
//   BROAD   the same, one group of up to 16 warps, whose registers hold no weights
// A CTA is as many warps as the registers hold, so that few partial rows are
// written and added: 16 with up to 16 columns a lane, 12 with up to 32, 8 if the
// generator is beside those.
//
// What bounds it: memory, where rows are long and many: bf16 with residual 131072 x
// 1600 241 us (1.03 of the measured copy rate: four fifths of the bytes are reads),
// 32768 x 4096 125 us (0.95), 65536 x 768 64 us (0.93), float32 16384 x 4096 134 us
// (0.89).  The split: up to 32 columns a lane keep the row's fixed costs (two sums,
// addresses) below a third of the instructions, and the column sums of them (64
// registers) still leave 12 warps; with one piece a lane and seven warps a row
// 131072 x 1600 took 420 us, with one warp and seven pieces 558.  With dropout it is
// latency: 131072 x 1600 414 us (0.75).  A piece takes about 260 instructions, a third
// of them the generator's and the selection's, in 238 registers; so 8 warps are on a
// multiprocessor, two a scheduler, each in its own chains of ten dependent rounds.
// Nothing is full: they issue in 49 % of the cycles, the multiply pipe is busy in 55 %,
// the memory gives 55 % of its peak.  Drawing the mask as bits before the row, by the
// same warp, which frees registers for 12 warps, took 475.  Calls of a few thousand rows
// are bound by the column sums' way out (through shared memory, a partial row a CTA, and
// a second kernel): 8192 x 768 takes 14.5 us from memory; with its data in L2 11.6,
// and 7.7 of them without the sums.  BROAD is short of registers (its 128 hold 64 of
// sums): 8192 x 16384 245 us (0.49).  Off the grid, 65536 x 1001 95 us (0.61).
enum BwdMode { NARROW, WIDE, BROAD };

__host__ __device__ constexpr int bwd_warps(int columns, BwdMode mode, bool drop) {
    return mode == BROAD || columns <= 16 ? 16 : drop ? 8 : 12;
}
// Rows of the ring: what the shared memory of a multiprocessor holds for them (a
// stage is 1536 C bytes a warp).
__host__ __device__ constexpr int bwd_ring_rows(int C, int columns, BwdMode mode, bool drop) {
    const int warps = bwd_warps(columns, mode, drop);
    return 3 * 1584 * C * warps <= kMaxRing ? 3 : 2 * 1584 * C * warps <= kMaxRing ? 2 : 1;
}

template <typename T, int C, BwdMode MODE, bool DROP, bool SHIFT>
__global__ void __launch_bounds__(bwd_warps(C * 16 / sizeof(T), MODE, DROP) * 32) ln_bwd_ring_kernel(const BwdParams<T> p, int team) {
    extern __shared__ uint4 s_ring[];  // [warp][stage][dy, r, dresidual][c][slot]; at the end the groups' column sums
    __shared__ float2 s_sum[2][16];
    constexpr int V = 16 / sizeof(T), H = V / 2, S = bwd_ring_rows(C, C * V, MODE, DROP);
    constexpr bool kKeepDev = SHIFT && sizeof(T) == 4;
    constexpr bool kHeld = MODE != BROAD, kCta = MODE != NARROW;  // weights in registers; otherwise from L1 in every row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    // NARROW: lanes a row, and each warp is a group; otherwise warps a row, and a group
    const int lanes = kCta || C > 1 ? 32 : team, group_warps = kCta ? team : 1;
    const int group = warp / group_warps, groups = nw / group_warps;
    // piece c of this thread is piece t + 32 c of its row: a warp's are adjacent
    const int t = kCta ? (warp - group * group_warps) * 32 * C + lane : lane & (lanes - 1);
    const int N = static_cast<int>(p.N), pieces = SHIFT ? (N + V - 1) / V : N / V;
    const float inv_n = 1.0f / static_cast<float>(N);
    const f32x2 zero2 = pair_of(0.0f, 0.0f);
    // whether this thread's piece c lies in the row: all but the last of a warp's do
    auto has = [&](int c) { return (!kCta && c < C - 1) || t + c * 32 < pieces; };
    uint4 carry = make_uint4(0, 0, 0, 0), carry_b = carry;
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

    f32x2 w[kHeld ? C : 1][H], dw[C][H], db[C][H];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < H; ++i) dw[c][i] = db[c][i] = zero2;
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < H; ++i) w[c][i] = zero2;
            if (has(c)) load_params2<T, V, SHIFT>(p.w, (t + c * 32) * V, N, w[c]);
        }
    }
    Philox g;
    if constexpr (DROP) g = Philox(p.drop.rng);
    const uint64_t first_m0 = kPhiloxM0 * static_cast<uint32_t>(t * (V / 4));

    const int rows_group = kCta ? 1 : 32 / lanes, rows_cta = rows_group * groups;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_cta;
    const int64_t base0 = static_cast<int64_t>(blockIdx.x) * rows_cta + group * rows_group;  // the group's first row
    const int sub = kCta ? 0 : lane / lanes;

    constexpr int kSlots = warp_slots(SHIFT, !kCta && C == 1), kStage = 3 * C * kSlots;
    uint4* const ring = s_ring + warp * (S * kStage) + lane + (SHIFT ? lane / lanes : 0);  // [stage][tensor][c][slot]
    const bool team_end = SHIFT && (kCta ? lane == 31 : t == lanes - 1);
    const uint32_t ring_at = smem_u32(ring);
    auto fill_tensor = [&](uint32_t to, const T* x, int64_t ld, int64_t row) {
        const T* start = x + row * ld;
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
    // the pieces of a row; nothing for a row past the last, which nothing is taken from
    auto fill = [&](int stage, int64_t row) {
        if (row < p.M) {
            const uint32_t to = ring_at + stage * kStage * 16;
            fill_tensor(to, p.dy, p.ld_dy, row);
            fill_tensor(to + C * kSlots * 16, p.r, p.ld_r, row);
            if (p.dres) fill_tensor(to + 2 * C * kSlots * 16, p.dres, p.ld_dres, row);
        }
        cp_async_commit();
    };
    if constexpr (!SHIFT) {  // pieces past the row are zeros in every stage, and stay so
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (!has(c))
                for (int k = 0; k < S * 3; ++k) ring[(k * C + c) * kSlots] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);
    float mean = base0 + sub < p.M ? p.mean[base0 + sub] : 0.0f;
    float rstd = base0 + sub < p.M ? p.rstd[base0 + sub] : 0.0f;
    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
    int buf = 0, stage = 0;
#pragma unroll 1
    for (int64_t base = base0; base < p.M; base += stride) {
        const int64_t row = base + sub, ahead = row + stride;
        const bool in = sub == 0 || row < p.M;  // (lanes of a warp that take several rows)
        const float mean_next = ahead < p.M ? p.mean[ahead] : 0.0f, rstd_next = ahead < p.M ? p.rstd[ahead] : 0.0f;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        cp_async_wait<S - 1>();
        uint4* const at = ring + stage * kStage;
        if constexpr (SHIFT) __syncwarp();
        const uint32_t mis_dy = SHIFT ? granule_offset(p.dy + row * p.ld_dy) : 0;
        const uint32_t mis_r = SHIFT ? granule_offset(p.r + row * p.ld_r) : 0;
        const uint32_t mis_dres = SHIFT && p.dres ? granule_offset(p.dres + row * p.ld_dres) : 0;
        const f32x2 shift = pair_of(-mean, -mean), scale = pair_of(rstd, rstd);
        // dy, the deviations r - mean, and g = dy * w (first pass) or g + less (second) of piece c.
        // SHIFT: the first pass cuts the pieces from the granules, without what is not the row's, and
        // leaves them (of float32 r the deviations: the second pass's own subtraction would cost 2999 x
        // 1237 18.6 us against 17.1) where its own granules were for the second
        auto inputs = [&](int c, bool first, f32x2 less, f32x2 (&dy)[H], f32x2 (&dev)[H], f32x2 (&gw)[H]) {
            Piece<T, V> a, b;
            uint4* const dy_slot = at + c * kSlots;
            uint4* const r_slot = at + (C + c) * kSlots;
            if (SHIFT && first) {
                a.raw = read_piece<T, true>(dy_slot, mis_dy);
                b.raw = read_piece<T, true>(r_slot, mis_r);
                __syncwarp();  // every lane has read its neighbour's granule
                const int valid = in ? count(c) : 0;
                if (valid < V) {
                    clear_from(a, valid);
                    clear_from(b, valid);
                }
                if constexpr (kKeepDev) {
                    unpack2(b, dev);
#pragma unroll
                    for (int i = 0; i < H; ++i) dev[i] = add2(dev[i], shift);
                    pack2(b, dev);
                }
                *dy_slot = a.raw;
                *r_slot = b.raw;
            } else {
                a.raw = *dy_slot;
                b.raw = *r_slot;
            }
            unpack2(a, dy);
            unpack2(b, dev);
            f32x2 wl[H];
            if constexpr (!kHeld) {
#pragma unroll
                for (int i = 0; i < H; ++i) wl[i] = zero2;
                if (has(c)) load_params2<T, V, SHIFT>(p.w, (t + c * 32) * V, N, wl);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const f32x2 weight = kHeld ? w[kHeld ? c : 0][i] : wl[i];
                if constexpr (!kKeepDev) dev[i] = add2(dev[i], shift);
                gw[i] = first ? mul2(dy[i], weight) : fma2(dy[i], weight, less);
            }
        };
        f32x2 c1v = zero2, c2v = zero2;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!SHIFT && C == 1 && !kCta && !in) continue;
            f32x2 dy[H], xhat[H], gw[H];  // pieces past the row: dy = 0, which adds nothing
            inputs(c, true, zero2, dy, xhat, gw);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                xhat[i] = mul2(xhat[i], scale);
                c1v = add2(c1v, gw[i]);
                c2v = fma2(gw[i], xhat[i], c2v);
                dw[c][i] = fma2(dy[i], xhat[i], dw[c][i]);
                db[c][i] = add2(db[c][i], dy[i]);
            }
        }
        const float2 h1 = split(c1v), h2 = split(c2v);
        float c1 = h1.x + h1.y, c2 = h2.x + h2.y;
        for (int o = lanes / 2; o; o >>= 1) {
            c1 += __shfl_xor_sync(0xFFFFFFFFu, c1, o);
            c2 += __shfl_xor_sync(0xFFFFFFFFu, c2, o);
        }
        if constexpr (kCta) {
            // two buffers: a warp that runs ahead writes the other one, and cannot reach this one
            // again before every warp of its group has passed the next row's barrier
            if (lane == 0) s_sum[buf][warp] = make_float2(c1, c2);
            if constexpr (MODE == BROAD) __syncthreads();
            else named_barrier(1 + group, group_warps * 32);
            c1 = c2 = 0.0f;
#pragma unroll 4
            for (int k = 0; k < group_warps; ++k) {
                const float2 f = s_sum[buf][group * group_warps + k];
                c1 += f.x;
                c2 += f.y;
            }
            buf ^= 1;
        }
        // (also keeps the compiler from carrying the first pass's values into the second, in more
        // registers than there are; where warps meet, their barrier does)
        if constexpr (!kCta) __syncwarp();
        // dr = rstd ((g - c1) + (r - mean) (-rstd c2)) + dres: four operations a column from dy on.
        // The deviation is formed before anything is multiplied by it, so a mean far above it costs no
        // digits, and rstd, which may be finite where its square is not (eps = 0), is never squared.
        const float slope = -rstd * (c2 * inv_n), less = -(c1 * inv_n);
        T* dx_row = p.dx + row * p.ld_dx;
        T* db_row = p.dbranch + row * p.ld_db;
        const f32x2 slope2 = pair_of(slope, slope), less2 = pair_of(less, less);
        uint64_t row_m0 = 0;
        if constexpr (DROP) row_m0 = g.row(static_cast<uint32_t>(row));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int valid = in && has(c) ? count(c) : 0;
            f32x2 dy[H], dev[H], d[H], rest[H];
            Piece<T, V> out;
            inputs(c, false, less2, dy, dev, d);
            if (p.dres) {
                out.raw = read_piece<T, SHIFT>(at + (2 * C + c) * kSlots, mis_dres);
                unpack2(out, rest);
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) rest[i] = zero2;
            }
#pragma unroll
            for (int i = 0; i < H; ++i) d[i] = fma2(fma2(dev[i], slope2, d[i]), scale, rest[i]);
            pack2(out, d);
            if constexpr (SHIFT) put(out.raw, carry, dx_row, c, valid);
            else if (valid > 0) out.store(dx_row + t * V + c * 32 * V);
            if (p.dbranch) {
                if constexpr (DROP) {
                    uint32_t words[V];
                    words_at<V>(g, first_m0 + kPhiloxM0 * static_cast<uint32_t>(c * 32 * (V / 4)), row_m0, words);
#pragma unroll
                    for (int i = 0; i < H; ++i) d[i] = dropped2(mul2(d[i], inv2), words[2 * i], words[2 * i + 1], p.drop);
                    pack2(out, d);
                }
                if constexpr (SHIFT) put(out.raw, carry_b, db_row, c, valid);
                else if (valid > 0) out.store(db_row + t * V + c * 32 * V);
            }
        }
        mean = mean_next;
        rstd = rstd_next;
        stage = stage == S - 1 ? 0 : stage + 1;
        if constexpr (SHIFT) __syncwarp();  // the granules that a neighbour read may be overwritten now
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
    if (p.part == nullptr) return;

    // The groups' sums to shared memory, where the ring was; their sum, in order, is the partial row.
    // Column i of a warp's piece (c, lane) is at [c][i][lane], rows kPitch floats apart: the lanes
    // write 32 banks, and 32 adjacent columns (V columns of 32 / V pieces) are read from 32 banks.
    constexpr int kPitch = 32 + 32 / V, kWarp = C * V * kPitch;
    __syncthreads();
    float* const s_part = reinterpret_cast<float*>(s_ring);  // [group][dw, db][warp of the group][c][i][lane]
    float* const own = s_part + (group * 2 * group_warps + warp - group * group_warps) * kWarp + lane;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 pw = split(dw[c][i / 2]), pb = split(db[c][i / 2]);
            float a = i & 1 ? pw.y : pw.x, b = i & 1 ? pb.y : pb.x;
            for (int o = lanes; o < 32; o *= 2) {  // lanes that took other rows of the same columns
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
            own[(c * V + i) * kPitch] = a;
            own[group_warps * kWarp + (c * V + i) * kPitch] = b;
        }
    }
    __syncthreads();
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
    for (int j = threadIdx.x; j < 2 * N; j += blockDim.x) {
        const int col = j < N ? j : j - N, piece = col / V;
        const int run = piece / 32;  // of the row: C runs a warp
        const float* from = s_part + ((j < N ? 0 : group_warps) + run / C) * kWarp + ((run % C) * V + col % V) * kPitch + piece % 32;
        float sum = from[0];
        for (int k = 1; k < groups; ++k) sum += from[k * 2 * group_warps * kWarp];
        if (gridDim.x > 1) {
            part[j] = sum;
        } else if (float* out = j < N ? p.dweight : p.dbias) {  // the one CTA's sums are the result
            out += col;
            *out = p.accumulate ? *out + sum : sum;
        }
    }
}

template <typename T, int C, BwdMode MODE, bool DROP, bool SHIFT>
cudaError_t launch_ring_as(BwdParams<T>& p, int team, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    // a row that fits WIDE's warps at these columns a lane goes there
    static_assert(MODE != BROAD || bwd_warps(C * V, WIDE, DROP) < 16, "no call reaches this variant");
    // groups (rows, or warps of narrow rows) a CTA: as many as fit, fewer where that leaves multiprocessors
    // idle -- but one CTA for what it takes at a time, whose sums need no second kernel
    const int warps = MODE == NARROW ? 1 : team;
    const int64_t rows = MODE == NARROW ? 32 / (C > 1 ? 32 : team) : 1;
    const int64_t all = (p.M + rows - 1) / rows;
    const int64_t most = std::max(1, bwd_warps(C * V, MODE, DROP) / warps);
    const int64_t groups = all <= most ? all : std::min<int64_t>(most, (all + sm_count() - 1) / sm_count());
    const unsigned block = static_cast<unsigned>(groups) * warps * 32;
    // one wave: as many CTAs as run at a time (kept by device and CTA size)
    static DeviceTable<17> table;
    const auto kern = ln_bwd_ring_kernel<T, C, MODE, DROP, SHIFT>;
    const size_t smem = size_t(bwd_ring_rows(C, C * V, MODE, DROP)) * 3 * C * (block / 32) * warp_slots(SHIFT, MODE == NARROW && C == 1) * 16;
    int n = 0;
    const cudaError_t e = resident_ctas(table, kern, block, smem, kMaxRing, &n);
    if (e != cudaSuccess) return e;
    p.parts = static_cast<int>(std::min<int64_t>({p.parts, int64_t(n) * sm_count(), (all + groups - 1) / groups}));
    return launch_pdl(kern, dim3(p.parts), dim3(block), smem, stream, p, team);
}

template <typename T, int C, BwdMode MODE, bool SHIFT>
cudaError_t launch_ring(BwdParams<T>& p, int team, cudaStream_t stream) {
    return p.drop.on && p.dbranch ? launch_ring_as<T, C, MODE, true, SHIFT>(p, team, stream)
                                  : launch_ring_as<T, C, MODE, false, SHIFT>(p, team, stream);
}

}  // namespace

// The one-pass kernels, where the row fits one; cudaErrorNotSupported where it
// does not.  Lowers p.parts to the partial rows that are written.
template <typename T, bool SHIFT>
cudaError_t launch_bwd_ring(BwdParams<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int64_t pieces = (p.N + V - 1) / V;
    const int team = team_of(pieces);
    switch ((pieces + team - 1) / team) {
        case 1: return launch_ring<T, 1, NARROW, SHIFT>(p, team, stream);
        case 2: return launch_ring<T, 2, NARROW, SHIFT>(p, team, stream);
        case 3: return launch_ring<T, 3, NARROW, SHIFT>(p, team, stream);
        case 4: return launch_ring<T, 4, NARROW, SHIFT>(p, team, stream);
        default: break;
    }
    const int warps = static_cast<int>((pieces + 127) / 128);  // of a row
    if (warps <= bwd_warps(4 * V, WIDE, p.drop.on && p.dbranch)) {
        // (two or three warps may do with three pieces a lane; more need the fourth)
        if (pieces <= 96 * warps) return launch_ring<T, 3, WIDE, SHIFT>(p, warps, stream);
        return launch_ring<T, 4, WIDE, SHIFT>(p, warps, stream);
    }
    if constexpr (V == 8) {
        if (warps <= 16) return launch_ring<T, 4, BROAD, SHIFT>(p, warps, stream);
    } else {  // (at four columns a piece WIDE takes 16 warps of four pieces; BROAD begins past it)
        if (pieces <= 16 * 256) return launch_ring<T, 8, BROAD, SHIFT>(p, static_cast<int>((pieces + 255) / 256), stream);
    }
    return cudaErrorNotSupported;
}

}  // namespace fp8q
