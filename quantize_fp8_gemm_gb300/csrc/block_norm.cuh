// block_norm.cuh -- the one-pass kernels of block_norm_fwd and block_norm_bwd, which
// block_norm.cu launches; each element type, on and off the 16-byte grid, is a
// translation unit of its own (block_norm_*.cu), so that they compile side by side.
#pragma once

#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>

namespace fp8q {

template <typename T>
struct BnFwd {
    int64_t M, N;
    const T* x;
    int64_t ldx;
    const T* res;
    int64_t ld_res;
    T* r_out;
    int64_t ld_r;
    T* y;
    int64_t ldy;
    Params<T> w, wp;       // of the norm before the next block; of the block's output
    const float* gate;     // [M] or NULL
    const float* alpha;    // or NULL: 1
    float* rstd;
    float* rstd_post;
    float eps;
    bool post, pre;        // norm after the block, norm before the next one
    QuantOut quant;
};

template <typename T>
struct BnBwd {
    int64_t M, N;
    const T* dy;           // NULL: no norm before the next block
    int64_t ld_dy;
    const T* r;
    int64_t ld_r;
    const T* dr;           // the stream's gradient on its other way, or NULL
    int64_t ld_dr;
    const T* x;            // NULL: nothing of the block's output is wanted
    int64_t ldx;
    const T* res;          // NULL unless dalpha is wanted
    int64_t ld_res;
    T* dres;
    int64_t ld_dres;
    T* dx;
    int64_t ld_dx;
    Params<T> w, wp;
    const float* gate;
    const float* alpha;
    const float* rstd;
    const float* rstd_post;
    float* dgate;
    float* part;           // [parts][2][N] sums of dw and dwp, then [parts] of dalpha; NULL: not wanted
    int parts;
    bool post;
};

namespace {

// Sum over the row of one value a thread: a team of lanes, or (CTA) all warps by one exchange
// through `s` (16 floats), in a fixed order.
template <bool CTA, bool PART>
__device__ __forceinline__ float row_sum(float v, int team, float* s, int warp, int lane, int nw) {
    v = team_sum<PART>(v, team);
    if constexpr (CTA) {
        if (lane == 0) s[warp] = v;
        __syncthreads();
        v = 0.0f;
        for (int k = 0; k < nw; ++k) v += s[k];
    }
    return v;
}

__device__ __forceinline__ float fold(f32x2 v) {
    const float2 f = split(v);
    return f.x + f.y;
}

// The forward: one pass over rows of 16-byte pieces, from a ring of rows in shared memory.
//   NARROW (CTA = false)  `team` lanes of a warp take a row, up to 64 columns a lane
//   CTA                   a CTA of up to 512 threads takes a row, 32 columns a thread
// The row stays in registers from its one read to its one write; its two sums of squares (of
// the block's output, and of the stored stream) are team shuffles, or an exchange each.
// Weights: in registers up to 32 columns a lane, in shared memory above.  S rows of the ring.
template <typename T, int C, bool CTA, bool SHIFT, int S>
__global__ void __launch_bounds__(CTA ? 512 : 128)
bn_fwd_kernel(const BnFwd<T> p, int team) {
    extern __shared__ uint4 s_ring[];
    __shared__ float s_sum[2][2][16];
    constexpr int V = 16 / sizeof(T), H = V / 2;
    constexpr bool kHeld = C * V <= 32;
    constexpr int kSlots = warp_slots(SHIFT, !CTA && C == 1), kStage = 2 * C * kSlots;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if constexpr (C > 1 || CTA) team = 32;
    const int t = CTA ? warp * 32 * C + lane : lane & (team - 1);  // piece c of this thread is piece t + 32 c
    const int N = static_cast<int>(p.N), pieces = (N + V - 1) / V;
    const float inv_n = 1.0f / static_cast<float>(N);
    const f32x2 zero2 = pair_of(0.0f, 0.0f);
    auto has = [&](int c) { return t + c * 32 < pieces; };
    auto count = [&](int c) { return SHIFT ? min(V, N - (t + c * 32) * V) : V; };
    uint4 carry = make_uint4(0, 0, 0, 0);
    auto put = [&](uint4 q, T* start, int c, int valid) {
        const bool head = c == 0 && (CTA ? lane : t) == 0, tail = t + c * 32 == pieces - 1 || (CTA && c == C - 1 && lane == 31);
        store_shifted<T, true, true>(q, carry, start, t + c * 32, valid, head, tail);
    };
    pdl_wait();

    // [w, wp][four columns of a piece][c][lane]
    float4* const s_par = reinterpret_cast<float4*>(s_ring + nw * (S * kStage)) + lane;
    f32x2 w[kHeld ? C : 1][H], wp[kHeld ? C : 1][H];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < H; ++i) w[c][i] = wp[c][i] = zero2;
            if (has(c)) {
                load_params2<T, V, SHIFT>(p.w, (t + c * 32) * V, N, w[c]);
                load_params2<T, V, SHIFT>(p.wp, (t + c * 32) * V, N, wp[c]);
            }
        } else if (warp == c % 4 && has(c)) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x2 f[H];
                load_params2<T, V, SHIFT>(q ? p.wp : p.w, (t + c * 32) * V, N, f);
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    const float2 a = split(f[2 * i]), b = split(f[2 * i + 1]);
                    s_par[((q * (V / 4) + i) * C + c) * 32] = make_float4(a.x, a.y, b.x, b.y);
                }
            }
        }
    }
    if constexpr (!kHeld) __syncthreads();
    auto weights = [&](int q, int c, f32x2 (&f)[H]) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < H; ++i) f[i] = q ? wp[c][i] : w[c][i];
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 v = s_par[((q * (V / 4) + i) * C + c) * 32];
                f[2 * i] = pair_of(v.x, v.y);
                f[2 * i + 1] = pair_of(v.z, v.w);
            }
        }
    };
    const float s = p.quant.on ? *p.quant.scale : 0.0f;
    const float alpha = p.alpha ? *p.alpha : 1.0f;
    uint32_t amax = 0, amax2 = 0, nsat = 0;

    const int rows_warp = CTA ? 1 : 32 / team, rows_cta = CTA ? 1 : rows_warp * nw;
    const uint32_t M = static_cast<uint32_t>(p.M), stride = gridDim.x * rows_cta, base0 = blockIdx.x * rows_cta;
    const uint32_t sub = CTA ? 0 : warp * rows_warp + lane / team;
    uint4* const ring = s_ring + warp * (S * kStage) + lane + (SHIFT ? lane / team : 0);  // [stage][x, residual][c][slot]
    const bool team_end = SHIFT && (CTA ? lane == 31 : t == team - 1);
    const uint32_t ring_at = smem_u32(ring);
    auto fill_tensor = [&](uint32_t to, const T* start) {
        const uint32_t mis = SHIFT ? granule_offset(start) : 0;
        const uint8_t* first = reinterpret_cast<const uint8_t*>(start) - mis;
        const int end = N * static_cast<int>(sizeof(T)) + static_cast<int>(mis);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (SHIFT) copy_granules<false>(to + c * kSlots * 16, first, t + c * 32, end, team_end);
            else if (has(c)) cp_async16(to + c * kSlots * 16, start + (t + c * 32) * V);
        }
    };
    auto fill = [&](int stage, uint32_t row) {  // nothing for a row past the last
        if (row < M) {
            const uint32_t to = ring_at + stage * kStage * 16;
            fill_tensor(to, p.x + row * p.ldx);
            if (p.res) fill_tensor(to + C * kSlots * 16, p.res + row * p.ld_res);
        }
        cp_async_commit();
    };
    if constexpr (!SHIFT) {  // pieces past the row are zeros in every stage, and stay so
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (!has(c))
                for (int k = 0; k < S * 2; ++k) ring[(k * C + c) * kSlots] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);

    float gate_next = 1.0f;  // read a row ahead
    if (p.gate && base0 + sub < M) gate_next = p.gate[base0 + sub];
    int stage = 0, buf = 0;
    for (uint32_t base = base0; base < M; base += stride) {
        const uint32_t row = base + sub;
        const bool in = row < M;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        const float gate = gate_next;
        if (p.gate && row + stride < M) gate_next = p.gate[row + stride];
        cp_async_wait<S - 1>();
        if constexpr (SHIFT) __syncwarp();
        const uint4* at = ring + stage * kStage;
        const uint32_t mis_x = SHIFT ? granule_offset(p.x + row * p.ldx) : 0;
        const uint32_t mis_r = SHIFT && p.res ? granule_offset(p.res + row * p.ld_res) : 0;
        auto clip = [&](int c, f32x2 (&v)[H]) {
            if constexpr (SHIFT) {
                if (!has(c) || count(c) < V) zero_from<V>(v, has(c) ? count(c) : 0);
            }
        };
        f32x2 v[C][H];
        f32x2 sq[2] = {zero2, zero2};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Piece<T, V> a;
            a.raw = read_piece<T, SHIFT>(at + c * kSlots, mis_x);
            unpack2(a, v[c]);
            clip(c, v[c]);
#pragma unroll
            for (int i = 0; i < H; ++i) sq[i & 1] = fma2(v[c][i], v[c][i], sq[i & 1]);
        }
        float rp = 1.0f;
        if (p.post) {
            const float sum = row_sum<CTA, C == 1 && !CTA>(fold(add2(sq[0], sq[1])), team, s_sum[buf][0], warp, lane, nw);
            rp = 1.0f / sqrtf(__fmaf_rn(sum, inv_n, p.eps));
            if (p.rstd_post && in && t == 0) p.rstd_post[row] = rp;
        }
        const f32x2 rp2 = pair_of(rp, rp), gate2 = pair_of(gate, gate), alpha2 = pair_of(alpha, alpha);
        sq[0] = sq[1] = zero2;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            f32x2 f[H];
            weights(1, c, f);
#pragma unroll
            for (int i = 0; i < H; ++i) v[c][i] = mul2(mul2(mul2(v[c][i], rp2), f[i]), gate2);
            if (p.res) {
                Piece<T, V> a;
                a.raw = read_piece<T, SHIFT>(at + (C + c) * kSlots, mis_r);
                f32x2 r[H];
                unpack2(a, r);
#pragma unroll
                for (int i = 0; i < H; ++i) v[c][i] = fma2(alpha2, r[i], v[c][i]);
            }
            Piece<T, V> a;
            pack2(a, v[c]);
            if (p.r_out) {
                const int valid = in && has(c) ? count(c) : 0;
                if constexpr (SHIFT) put(a.raw, p.r_out + row * p.ld_r, c, valid);
                else if (valid) a.store(p.r_out + row * p.ld_r + (t + c * 32) * V);
            }
            unpack2(a, v[c]);
            if (!SHIFT && !has(c)) {
#pragma unroll
                for (int i = 0; i < H; ++i) v[c][i] = zero2;
            }
            clip(c, v[c]);
#pragma unroll
            for (int i = 0; i < H; ++i) sq[i & 1] = fma2(v[c][i], v[c][i], sq[i & 1]);
        }
        if (p.pre) {
            const float sum = row_sum<CTA, C == 1 && !CTA>(fold(add2(sq[0], sq[1])), team, s_sum[buf][1], warp, lane, nw);
            const float rstd = 1.0f / sqrtf(__fmaf_rn(sum, inv_n, p.eps));
            if (p.rstd && in && t == 0) p.rstd[row] = rstd;
            const f32x2 rstd2 = pair_of(rstd, rstd);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int valid = in && has(c) ? count(c) : 0;
                if (!SHIFT && valid == 0) continue;
                f32x2 f[H];
                weights(0, c, f);
#pragma unroll
                for (int i = 0; i < H; ++i) v[c][i] = mul2(mul2(v[c][i], rstd2), f[i]);
                Piece<T, V> y;
                pack2(y, v[c]);
                if (p.y) {
                    if constexpr (SHIFT) put(y.raw, p.y + row * p.ldy, c, valid);
                    else y.store(p.y + row * p.ldy + (t + c * 32) * V);
                }
                if (p.quant.on && valid > 0) {
                    uint8_t* dst = p.quant.q ? p.quant.q + row * p.N + (t + c * 32) * V : nullptr;
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
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        buf ^= 1;
        if constexpr (SHIFT) __syncwarp();  // the granules that a neighbour read may be overwritten now
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
    if (p.quant.on) publish_quant(p.quant, max(amax, max16x2(amax2) << 16), nsat);
}

template <typename T, int C, bool CTA, bool SHIFT, int S = 3>
cudaError_t launch_bn_fwd_as(const BnFwd<T>& p, int team, unsigned block, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    static DeviceTable<17> table;
    const auto kern = bn_fwd_kernel<T, C, CTA, SHIFT, S>;
    size_t smem = size_t(S) * 2 * C * (block / 32) * warp_slots(SHIFT, !CTA && C == 1) * 16;
    if (C * V > 32) smem += size_t(2) * C * 32 * V * sizeof(float);
    int n = 0;
    const cudaError_t e = resident_ctas(table, kern, block, smem, kMaxRing, &n);
    if (e != cudaSuccess) return e;
    const int64_t rows = CTA ? 1 : 128 / team;
    const int64_t grid = std::min<int64_t>((p.M + rows - 1) / rows, int64_t(n) * sm_count());
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, p, team);
}

// The backward: `team` lanes of a warp (NARROW, up to 2 pieces a lane), or a group of warps
// (WIDE, 2 pieces a lane) take a row; a CTA is several warps or groups.  A thread keeps its
// columns' weights and sums for all its rows.
//     rhat = r rstd, g = dy w;  dr = dr_in + rstd (g - rhat sum(g rhat) / N)
//     xhat = x rstd_post;       e = sum(dr wp xhat)
//     dx = gate rstd_post (dr wp - xhat e / N)  [post],  gate dr wp  [not post]
// The row's inputs come through a ring of rows in shared memory: three, or two where the
// residual is read too.
constexpr int bn_bwd_stages(bool alpha) { return alpha ? 2 : 3; }
enum { IN_DY, IN_R, IN_DR, IN_X, IN_RES };

template <typename T, int C, bool WIDE, bool ALPHA, bool SHIFT>
__global__ void __launch_bounds__(512, 1)
bn_bwd_kernel(const BnBwd<T> p, int team) {
    extern __shared__ uint4 s_ring[];
    __shared__ float s_sum[2][2][16];
    constexpr int V = 16 / sizeof(T), H = V / 2, S = bn_bwd_stages(ALPHA), TENSORS = ALPHA ? 5 : 4;
    constexpr int kSlots = warp_slots(SHIFT, !WIDE && C == 1), kStage = TENSORS * C * kSlots;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    // WIDE: team = warps of a group; otherwise lanes of a row
    const int group = WIDE ? warp / team : warp, wg = WIDE ? warp - group * team : 0;
    const int lanes = WIDE || C > 1 ? 32 : team;
    const int t = WIDE ? wg * 32 * C + lane : lane & (lanes - 1);
    const int N = static_cast<int>(p.N), pieces = (N + V - 1) / V;
    const float inv_n = 1.0f / static_cast<float>(N);
    const f32x2 zero2 = pair_of(0.0f, 0.0f);
    auto has = [&](int c) { return t + c * 32 < pieces; };
    auto count = [&](int c) { return SHIFT ? min(V, N - (t + c * 32) * V) : V; };
    uint4 carry = make_uint4(0, 0, 0, 0);
    auto put = [&](uint4 q, T* start, int c, int valid) {
        const bool head = c == 0 && (WIDE ? lane : t) == 0, tail = t + c * 32 == pieces - 1 || (WIDE && c == C - 1 && lane == 31);
        store_shifted<T, true, true>(q, carry, start, t + c * 32, valid, head, tail);
    };
    pdl_wait();
    f32x2 w[C][H], wp[C][H], dw[C][H], dwp[C][H];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < H; ++i) w[c][i] = wp[c][i] = dw[c][i] = dwp[c][i] = zero2;
        if (has(c)) {
            load_params2<T, V, SHIFT>(p.w, (t + c * 32) * V, N, w[c]);
            load_params2<T, V, SHIFT>(p.wp, (t + c * 32) * V, N, wp[c]);
        }
    }
    const float alpha = p.alpha ? *p.alpha : 1.0f;
    f32x2 dalpha2 = zero2;

    const int groups = WIDE ? nw / team : nw, rows_warp = WIDE ? 1 : 32 / lanes, rows_cta = groups * rows_warp;
    const uint32_t M = static_cast<uint32_t>(p.M), stride = gridDim.x * rows_cta, base0 = blockIdx.x * rows_cta;
    const uint32_t sub = group * rows_warp + (WIDE ? 0 : lane / lanes);
    uint4* const ring = s_ring + warp * (S * kStage) + lane + (SHIFT && !WIDE ? lane / lanes : 0);
    const bool team_end = SHIFT && (WIDE ? lane == 31 : t == lanes - 1);
    const uint32_t ring_at = smem_u32(ring);
    auto fill_tensor = [&](uint32_t to, const T* base, int64_t at) {
        if (base == nullptr) return;
        const T* start = base + at;
        const uint32_t mis = SHIFT ? granule_offset(start) : 0;
        const uint8_t* first = reinterpret_cast<const uint8_t*>(start) - mis;
        const int end = N * static_cast<int>(sizeof(T)) + static_cast<int>(mis);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (SHIFT) copy_granules<false>(to + c * kSlots * 16, first, t + c * 32, end, team_end);
            else if (has(c)) cp_async16(to + c * kSlots * 16, start + (t + c * 32) * V);
        }
    };
    auto fill = [&](int stage, uint32_t row) {
        if (row < M) {
            const uint32_t to = ring_at + stage * kStage * 16, step = C * kSlots * 16;
            fill_tensor(to + IN_DY * step, p.dy, row * p.ld_dy);
            if (p.dy) fill_tensor(to + IN_R * step, p.r, row * p.ld_r);
            fill_tensor(to + IN_DR * step, p.dr, row * p.ld_dr);
            fill_tensor(to + IN_X * step, p.x, row * p.ldx);
            if constexpr (ALPHA) fill_tensor(to + IN_RES * step, p.res, row * p.ld_res);
        }
        cp_async_commit();
    };
    if constexpr (!SHIFT) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (!has(c))
                for (int k = 0; k < S * TENSORS; ++k) ring[(k * C + c) * kSlots] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);

    auto group_sum = [&](float v, float* s) {
        v = team_sum<C == 1 && !WIDE>(v, lanes);
        if constexpr (WIDE) {
            if (lane == 0) s[warp] = v;
            named_barrier(1 + group, team * 32);
            v = 0.0f;
            for (int k = 0; k < team; ++k) v += s[group * team + k];
        }
        return v;
    };
    // a row's gate and statistics, read a row ahead
    float gate_next = 1.0f, rp_next = 1.0f, rs_next = 0.0f;
    auto scalars = [&](uint32_t row) {
        if (row >= M) return;
        if (p.gate) gate_next = p.gate[row];
        if (p.rstd_post) rp_next = p.rstd_post[row];
        if (p.dy) rs_next = p.rstd[row];
    };
    scalars(base0 + sub);
    int stage = 0, buf = 0;
    // (a group, or a warp with one row, is done at its own last row; lanes of several rows together)
    for (uint32_t base = base0; (WIDE || C > 1 ? base + sub : base) < M; base += stride) {
        const uint32_t row = base + sub;
        const bool in = row < M;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        const float gate = gate_next, rp = rp_next, rs = rs_next;
        scalars(row + stride);
        cp_async_wait<S - 1>();
        if constexpr (SHIFT) __syncwarp();
        const uint4* at = ring + stage * kStage;
        auto read = [&](int which, const T* base_p, int64_t off, int c, f32x2 (&v)[H]) {
            if (base_p == nullptr) {
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = zero2;
                return;
            }
            Piece<T, V> a;
            a.raw = read_piece<T, SHIFT>(at + (which * C + c) * kSlots, SHIFT ? granule_offset(base_p + off) : 0);
            unpack2(a, v);
            if constexpr (SHIFT) {
                if (!has(c) || count(c) < V) zero_from<V>(v, has(c) ? count(c) : 0);
            }
        };
        f32x2 dr[C][H];
        // the norm before the next block
        if (p.dy) {
            const f32x2 rs2 = pair_of(rs, rs);
            f32x2 rhat[C][H], acc[2] = {zero2, zero2};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 dy[H];
                read(IN_DY, p.dy, row * p.ld_dy, c, dy);
                read(IN_R, p.r, row * p.ld_r, c, rhat[c]);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    rhat[c][i] = mul2(rhat[c][i], rs2);
                    if (in) dw[c][i] = fma2(dy[i], rhat[c][i], dw[c][i]);
                    dr[c][i] = mul2(dy[i], w[c][i]);
                    acc[i & 1] = fma2(dr[c][i], rhat[c][i], acc[i & 1]);
                }
            }
            const float along = -group_sum(fold(add2(acc[0], acc[1])), s_sum[buf][0]) * inv_n;
            const f32x2 along2 = pair_of(along, along);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 d[H];
                read(IN_DR, p.dr, row * p.ld_dr, c, d);
#pragma unroll
                for (int i = 0; i < H; ++i) dr[c][i] = fma2(fma2(rhat[c][i], along2, dr[c][i]), rs2, d[i]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) read(IN_DR, p.dr, row * p.ld_dr, c, dr[c]);
        }
        if constexpr (ALPHA) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 f[H];
                read(IN_RES, p.res, row * p.ld_res, c, f);
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (in) dalpha2 = fma2(dr[c][i], f[i], dalpha2);
            }
        }
        if (p.dres) {
            const f32x2 alpha2 = pair_of(alpha, alpha);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 f[H];
#pragma unroll
                for (int i = 0; i < H; ++i) f[i] = mul2(dr[c][i], alpha2);
                Piece<T, V> a;
                pack2(a, f);
                const int valid = in && has(c) ? count(c) : 0;
                if constexpr (SHIFT) put(a.raw, p.dres + row * p.ld_dres, c, valid);
                else if (valid) a.store(p.dres + row * p.ld_dres + (t + c * 32) * V);
            }
        }
        // the block's output, its norm and its gate
        if (p.x) {
            const f32x2 rp2 = pair_of(rp, rp), gate2 = pair_of(gate, gate);
            f32x2 xhat[C][H], acc[2] = {zero2, zero2};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                read(IN_X, p.x, row * p.ldx, c, xhat[c]);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    xhat[c][i] = mul2(xhat[c][i], rp2);
                    if (in) dwp[c][i] = fma2(mul2(dr[c][i], gate2), xhat[c][i], dwp[c][i]);
                    dr[c][i] = mul2(dr[c][i], wp[c][i]);
                    acc[i & 1] = fma2(dr[c][i], xhat[c][i], acc[i & 1]);
                }
            }
            float along = 0.0f;
            if (p.post || p.dgate) {
                along = group_sum(fold(add2(acc[0], acc[1])), s_sum[buf][1]);
                if (p.dgate && in && t == 0) p.dgate[row] = along;
            }
            if (p.dx) {
                const float a1 = p.post ? -along * inv_n : 0.0f;
                const f32x2 along2 = pair_of(a1, a1);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    f32x2 f[H];
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        f[i] = p.post ? mul2(fma2(xhat[c][i], along2, dr[c][i]), rp2) : dr[c][i];
                        f[i] = mul2(f[i], gate2);
                    }
                    Piece<T, V> a;
                    pack2(a, f);
                    const int valid = in && has(c) ? count(c) : 0;
                    if constexpr (SHIFT) put(a.raw, p.dx + row * p.ld_dx, c, valid);
                    else if (valid) a.store(p.dx + row * p.ld_dx + (t + c * 32) * V);
                }
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        buf ^= 1;
        if constexpr (SHIFT) __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
    pdl_launch_dependents();
    if (p.part == nullptr) return;

    // the CTA's sums in shared memory: [warp or group][dw, dwp][columns], added in order
    float* const s_part = reinterpret_cast<float*>(s_ring);
    const int columns = WIDE ? team * 32 * C * V : 32 * C * V;  // of a group's (warp's) lanes
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int at = ((WIDE ? wg * 32 * C : 0) + lane + c * 32) * V + 2 * i;
            const float2 a = split(dw[c][i]), b = split(dwp[c][i]);
            float* d = s_part + group * 2 * columns;
            d[at] = a.x;
            d[at + 1] = a.y;
            d[columns + at] = b.x;
            d[columns + at + 1] = b.y;
        }
    __syncthreads();
    float* const out = p.part + int64_t(blockIdx.x) * 2 * p.N;
    // (NARROW with several rows a warp: each team of lanes holds sums of all columns)
    const int teams = WIDE ? 1 : 32 / lanes, width = WIDE || C > 1 ? columns : lanes * V;
    for (int j = threadIdx.x; j < N; j += blockDim.x) {
        float a = 0.0f, b = 0.0f;
        for (int g = 0; g < groups; ++g)
            for (int k = 0; k < teams; ++k) {
                a += s_part[g * 2 * columns + k * width + j];
                b += s_part[g * 2 * columns + columns + k * width + j];
            }
        out[j] = a;
        out[p.N + j] = b;
    }
    if constexpr (ALPHA) {
        float a = team_sum<false>(fold(dalpha2), 32);
        if (lane == 0) s_sum[0][0][warp] = a;
        __syncthreads();
        if (threadIdx.x == 0) {
            a = 0.0f;
            for (int k = 0; k < nw; ++k) a += s_sum[0][0][k];
            p.part[int64_t(p.parts) * 2 * p.N + blockIdx.x] = a;
        }
    }
}

template <typename T, int C, bool WIDE, bool ALPHA, bool SHIFT>
cudaError_t launch_bn_bwd_as(BnBwd<T> p, int team, unsigned block, int most, int* parts, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    static DeviceTable<17> table;
    const auto kern = bn_bwd_kernel<T, C, WIDE, ALPHA, SHIFT>;
    const int warps = block / 32;
    const size_t ring = size_t(bn_bwd_stages(ALPHA)) * (ALPHA ? 5 : 4) * C * warps * warp_slots(SHIFT, !WIDE && C == 1) * 16;
    const size_t sums = size_t(warps) * 2 * 32 * C * V * sizeof(float);
    const size_t smem = std::max(ring, sums);
    int n = 0;
    const cudaError_t e = resident_ctas(table, kern, block, smem, kMaxRing, &n);
    if (e != cudaSuccess) return e;
    const int64_t rows = WIDE ? warps / team : warps * (C > 1 ? 1 : 32 / team);
    const int64_t grid = std::min<int64_t>(std::min<int64_t>((p.M + rows - 1) / rows, int64_t(n) * sm_count()), most);
    p.parts = *parts = static_cast<int>(grid);
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, p, team);
}

}  // namespace

// The one-pass kernels, where the row fits one; cudaErrorNotSupported where it does not.
template <typename T, bool SHIFT>
cudaError_t launch_bn_fwd(const BnFwd<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), kMost = 32 / V;
    const int64_t pieces = (p.N + V - 1) / V;
    const int team = team_of(pieces);
    switch ((pieces + team - 1) / team) {
        case 1: return launch_bn_fwd_as<T, 1, false, SHIFT>(p, team, 128, stream);
        case 2: return launch_bn_fwd_as<T, 2, false, SHIFT>(p, team, 128, stream);
        case 3: return launch_bn_fwd_as<T, 3, false, SHIFT>(p, team, 128, stream);
        case 4: return launch_bn_fwd_as<T, 4, false, SHIFT>(p, team, 128, stream);
        case 5: return launch_bn_fwd_as<T, 5, false, SHIFT>(p, team, 128, stream);
        case 6: return launch_bn_fwd_as<T, 6, false, SHIFT>(p, team, 128, stream);
        case 7: return launch_bn_fwd_as<T, 7, false, SHIFT>(p, team, 128, stream);
        case 8: return launch_bn_fwd_as<T, 8, false, SHIFT>(p, team, 128, stream);
        default: break;
    }
    const unsigned block = threads_of(pieces, kMost);
    // three rows of 16 384 two-byte columns, or 8192 of four bytes, fit shared memory; of wider ones of four bytes one
    if (block <= (V == 8 ? 512 : 256)) return launch_bn_fwd_as<T, kMost, true, SHIFT>(p, 32, block, stream);
    if constexpr (V == 4)
        if (block <= 512) return launch_bn_fwd_as<T, kMost, true, SHIFT, 1>(p, 32, block, stream);
    return cudaErrorNotSupported;
}

// At most `most` partial rows; *parts of them are written.
template <typename T, bool ALPHA, bool SHIFT>
cudaError_t launch_bn_bwd(const BnBwd<T>& p, int most, int* parts, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), kC = 2;  // pieces a lane
    const int64_t pieces = (p.N + V - 1) / V;
    if (pieces <= 32) return launch_bn_bwd_as<T, 1, false, ALPHA, SHIFT>(p, team_of(pieces), 256, most, parts, stream);
    if (pieces <= 32 * kC) return launch_bn_bwd_as<T, kC, false, ALPHA, SHIFT>(p, 32, 512, most, parts, stream);
    const int64_t team = (pieces + 32 * kC - 1) / (32 * kC);
    if (team <= 16) {
        const unsigned block = static_cast<unsigned>(16 / team * team) * 32;
        return launch_bn_bwd_as<T, kC, true, ALPHA, SHIFT>(p, static_cast<int>(team), block, most, parts, stream);
    }
    return cudaErrorNotSupported;
}

}  // namespace fp8q
