// norm_fwd.cu -- layer_norm_fwd: dropout + residual addition + layer norm +
// FP8 cast in one launch.
//
//     d    = keep ? float32(x * inv) : 0            (p > 0)
//     r    = T(float32(residual + d))               -> r_out
//     mean = sum r / N,  var = sum (r - mean)^2 / N, rstd = 1 / sqrt(var + eps)
//     y    = T((r - mean) * rstd * w + b)
//     q    = FP8(float32(y * s)), max |y|, #{|y s| > max}
//
// The norm is that of the r which is stored, rounded to T: layer_norm_bwd
// reads that r, so its gradient is the gradient of what was computed, and the
// fused call equals dropout_fwd followed by a plain layer_norm_fwd bit for bit.
// Statistics are float32 sums of the deviations, not of squares, so a mean far
// above the deviation costs no digits.
#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace fp8q {

__global__ void clear_quant_kernel(float* amax, unsigned long long* sat) {
    pdl_launch_dependents();
    pdl_wait();
    if (amax) *amax = 0.0f;
    if (sat) *sat = 0ull;
}

namespace {

constexpr int kRing = 3;  // rows of the ring: one in use, two in flight

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

// Any width: one CTA per row, three passes over the row (the second and third
// from L1 / L2), each thread taking quads of columns (one generator block).
// The row is formed again from its inputs in every pass and r_out is written
// in the last, so r_out and y may replace an input.
template <typename T>
__device__ __forceinline__ void row_quad(const FwdParams<T>& p, int64_t row, int64_t quad, float (&r)[4]) {
    const int64_t j0 = quad * 4;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (p.drop.on) w = Philox(p.drop.rng).block(static_cast<uint32_t>(quad), static_cast<uint32_t>(row));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = 0.0f;
        if (j0 + i >= p.N) continue;
        float v = to_f32(p.x[row * p.ldx + j0 + i]);
        if (p.drop.on) v = dropped(v, word_of(w, i), p.drop);
        if (p.res) v = __fadd_rn(to_f32(p.res[row * p.ld_res + j0 + i]), v);
        r[i] = (p.drop.on || p.res) ? round_to<T>(v) : v;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) ln_fwd_loop_kernel(const FwdParams<T> p) {
    __shared__ float s_sum[66];
    pdl_wait();
    const int64_t quads = (p.N + 3) / 4;
    const float inv_n = 1.0f / static_cast<float>(p.N);
    uint32_t amax = 0, nsat = 0;
    const float s = p.quant.on ? *p.quant.scale : 0.0f;
    const float fmax = fp8_max_value(p.quant.fmt);
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        float r[4], sum = 0.0f, dev = 0.0f;
        for (int64_t q = threadIdx.x; q < quads; q += blockDim.x) {
            row_quad(p, row, q, r);
            sum += (r[0] + r[1]) + (r[2] + r[3]);
        }
        const float mean = block_sum2(sum, 0.0f, s_sum).x * inv_n;
        for (int64_t q = threadIdx.x; q < quads; q += blockDim.x) {
            row_quad(p, row, q, r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q * 4 + i < p.N) dev += (r[i] - mean) * (r[i] - mean);
        }
        const float rstd = 1.0f / sqrtf(block_sum2(dev, 0.0f, s_sum).x * inv_n + p.eps);
        for (int64_t q = threadIdx.x; q < quads; q += blockDim.x) {
            row_quad(p, row, q, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t j = q * 4 + i;
                if (j >= p.N) continue;
                if (p.r_out) p.r_out[row * p.ld_r + j] = from_f32<T>(r[i]);
                const T y = from_f32<T>((r[i] - mean) * rstd * p.w.at(j) + p.b.at(j));
                if (p.y) p.y[row * p.ldy + j] = y;
                if (p.quant.on) {
                    const float yf = to_f32(y), v = __fmul_rn(yf, s);
                    amax = max(amax, __float_as_uint(fabsf(yf)));
                    nsat += fabsf(v) > fmax;
                    if (p.quant.q) p.quant.q[row * p.N + j] = static_cast<uint8_t>(cast_pair(v, 0.0f, p.quant.fmt));
                }
            }
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
    }
    pdl_launch_dependents();
    if (p.quant.on) publish_quant(p.quant, amax, nsat);
}

// Rows of up to C pieces a thread, held in registers: one read of every input,
// one write of every output.  WIDE = false: `team` (a power of two <= 32) lanes
// of a warp take a row, statistics by shuffles.  WIDE = true: a CTA takes a row;
// each warp forms the mean and the squared deviations of its part, and the
// parts are joined in one exchange:  mean = sum n_w mean_w / N,
// sum dev^2 = sum (dev^2_w + n_w (mean_w - mean)^2).
template <typename T, int V, int C, bool DROP, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : 128)
ln_fwd_rows_kernel(const FwdParams<T> p, int team) {
    __shared__ float s_mean[32], s_dev[32], s_n[32];
    const int lane = threadIdx.x & 31;
    const int t = WIDE ? threadIdx.x : lane & (team - 1);  // this thread's place in its row's team
    const int64_t row = WIDE ? blockIdx.x : (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / team;
    const int span = WIDE ? blockDim.x : team;
    const int pieces = static_cast<int>(p.N / V);
    const bool in = row < p.M;
    const float inv_n = 1.0f / static_cast<float>(p.N);
    pdl_wait();

    float v[C][V];
    float sum = 0.0f;
    {
        Piece<T, V> a[C], r[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t + c * span;
            a[c].zero();
            if (in && k < pieces) a[c].load(p.x + row * p.ldx + static_cast<int64_t>(k) * V);
        }
        if (p.res) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = t + c * span;
                r[c].zero();
                if (in && k < pieces) r[c].load(p.res + row * p.ld_res + static_cast<int64_t>(k) * V);
            }
        }
        Philox g;
        if constexpr (DROP) g = Philox(p.drop.rng);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t + c * span;
            a[c].unpack(v[c]);
            if (DROP || p.res) {
                if constexpr (DROP) {
                    uint32_t w[V];
                    words_at<V>(g, static_cast<uint32_t>(k) * V, static_cast<uint32_t>(row), w);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[c][i] = dropped(v[c][i], w[i], p.drop);
                }
                if (p.res) {
                    float f[V];
                    r[c].unpack(f);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[c][i] = __fadd_rn(f[i], v[c][i]);
                }
                a[c].pack(v[c]);
                if (p.r_out && in && k < pieces) a[c].store(p.r_out + row * p.ld_r + static_cast<int64_t>(k) * V);
                a[c].unpack(v[c]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[c][i];  // pieces past the row are zeros
        }
    }

    int own = 0;  // elements of this thread
#pragma unroll
    for (int c = 0; c < C; ++c) own += t + c * span < pieces ? V : 0;
    int n = own;
    const int width = WIDE ? 32 : team;
    for (int o = width / 2; o; o >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (WIDE) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    }
    float mean = WIDE ? sum / static_cast<float>(max(n, 1)) : sum * inv_n;
    float dev = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (t + c * span < pieces) {
#pragma unroll
            for (int i = 0; i < V; ++i) dev = __fmaf_rn(v[c][i] - mean, v[c][i] - mean, dev);
        }
    }
    for (int o = width / 2; o; o >>= 1) dev += __shfl_xor_sync(0xFFFFFFFFu, dev, o);
    if constexpr (WIDE) {
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        if (lane == 0) {
            s_mean[warp] = mean;
            s_dev[warp] = dev;
            s_n[warp] = static_cast<float>(n);
        }
        __syncthreads();
        const float wn = lane < nw ? s_n[lane] : 0.0f, wm = lane < nw ? s_mean[lane] : 0.0f;
        dev = lane < nw ? s_dev[lane] : 0.0f;
        sum = wn * wm;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        mean = sum * inv_n;
        dev = __fmaf_rn(wn * (wm - mean), wm - mean, dev);
#pragma unroll
        for (int o = 16; o; o >>= 1) dev += __shfl_xor_sync(0xFFFFFFFFu, dev, o);
    }
    const float rstd = 1.0f / sqrtf(__fmaf_rn(dev, inv_n, p.eps));

    uint32_t amax = 0, nsat = 0;
    const float s = p.quant.on ? *p.quant.scale : 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = t + c * span;
        if (!in || k >= pieces) continue;
        const int64_t j = static_cast<int64_t>(k) * V;
        float w[V], b[V];
        load_params<T, V>(p.w, j, w);
        load_params<T, V>(p.b, j, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] = __fmaf_rn((v[c][i] - mean) * rstd, w[i], b[i]);
        Piece<T, V> y;
        y.pack(v[c]);
        if (p.y) y.store(p.y + row * p.ldy + j);
        if (p.quant.on) quant_piece<T, V>(p.quant, s, y, p.quant.q ? p.quant.q + row * p.N + j : nullptr, amax, nsat);
    }
    if (in && t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    pdl_launch_dependents();
    if (p.quant.on) publish_quant(p.quant, amax, nsat);
}

// Rows of 16-byte pieces, up to 16 columns a thread of a CTA (WIDE) or up to 64
// of a lane of a warp (NARROW).  One wave of CTAs takes rows in turn; each keeps
// its columns' weights and biases in registers and the next rows' pieces in
// flight in a ring of S rows in shared memory (a thread copies and reads its own
// pieces: it waits for its own copies, no barrier guards the ring).
template <typename T, int V, int C, bool DROP, bool RES, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 512 : 128) ln_fwd_ring_kernel(const FwdParams<T> p, int team) {
    extern __shared__ uint4 s_ring[];  // [stage][x, residual][c][thread]
    __shared__ float s_mean[2][16], s_dev[2][16], s_n[16];
    constexpr int S = kRing, H = V / 2, TENSORS = RES ? 2 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int t = WIDE ? threadIdx.x : lane & (team - 1);
    const int span = WIDE ? blockDim.x : team;
    const int pieces = static_cast<int>(p.N / V);
    const float inv_n = 1.0f / static_cast<float>(p.N);
    pdl_wait();

    f32x2 w[C][H], b[C][H];
    int own = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float f[V];
#pragma unroll
        for (int i = 0; i < H; ++i) w[c][i] = b[c][i] = pair_of(0.0f, 0.0f);
        if (t + c * span >= pieces) continue;
        own += V;
        load_params<T, V>(p.w, static_cast<int64_t>(t + c * span) * V, f);
#pragma unroll
        for (int i = 0; i < H; ++i) w[c][i] = pair_of(f[2 * i], f[2 * i + 1]);
        load_params<T, V>(p.b, static_cast<int64_t>(t + c * span) * V, f);
#pragma unroll
        for (int i = 0; i < H; ++i) b[c][i] = pair_of(f[2 * i], f[2 * i + 1]);
    }
    float inv_own = inv_n;  // 1 / (elements whose mean a warp forms)
    if constexpr (WIDE) {
        const int n = __reduce_add_sync(0xFFFFFFFFu, own);
        inv_own = n ? 1.0f / static_cast<float>(n) : 0.0f;
        if (lane == 0) s_n[warp] = static_cast<float>(n);  // read after the first row's barrier
    }
    Philox g;
    if constexpr (DROP) g = Philox(p.drop.rng);
    const float s = p.quant.on ? *p.quant.scale : 0.0f;
    uint32_t amax = 0, amax2 = 0, nsat = 0;

    const int rows_warp = WIDE ? 1 : 32 / team, rows_cta = WIDE ? 1 : rows_warp * nw;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_cta;
    const int64_t base0 = static_cast<int64_t>(blockIdx.x) * rows_cta;
    const int64_t sub = WIDE ? 0 : warp * rows_warp + lane / team;
    auto slot = [&](int stage, int tensor, int c) {
        return s_ring + ((stage * TENSORS + tensor) * C + c) * static_cast<int>(blockDim.x) + threadIdx.x;
    };
    // pieces past the row, and rows past the last, are zeros
    auto fill = [&](int stage, int64_t row) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool in = row < p.M && t + c * span < pieces;
            const int64_t j = static_cast<int64_t>(t + c * span) * V;
            cp_async16_or_zero(smem_u32(slot(stage, 0, c)), in ? p.x + row * p.ldx + j : p.x, in);
            if constexpr (RES)
                cp_async16_or_zero(smem_u32(slot(stage, 1, c)), in ? p.res + row * p.ld_res + j : p.res, in);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);

    int stage = 0, buf = 0;
    for (int64_t base = base0; base < p.M; base += stride) {
        const int64_t row = base + sub;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        cp_async_wait<S - 1>();
        f32x2 v[C][H], sum2 = pair_of(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t + c * span;
            Piece<T, V> a;
            a.raw = *slot(stage, 0, c);
            if constexpr (DROP || RES) {
                float f[V];
                a.unpack(f);
                if constexpr (DROP) {
                    uint32_t words[V];
                    words_at<V>(g, static_cast<uint32_t>(k) * V, static_cast<uint32_t>(row), words);
#pragma unroll
                    for (int i = 0; i < V; ++i) f[i] = dropped(f[i], words[i], p.drop);
                }
                if constexpr (RES) {
                    Piece<T, V> r;
                    r.raw = *slot(stage, 1, c);
                    unpack2(r, v[c]);
#pragma unroll
                    for (int i = 0; i < H; ++i) v[c][i] = add2(v[c][i], pair_of(f[2 * i], f[2 * i + 1]));
                    pack2(a, v[c]);
                } else {
                    a.pack(f);
                }
                if (p.r_out && row < p.M && k < pieces) a.store(p.r_out + row * p.ld_r + static_cast<int64_t>(k) * V);
            }
            unpack2(a, v[c]);
            f32x2 part = add2(v[c][0], v[c][1]);
            if constexpr (H == 4) part = add2(part, add2(v[c][2], v[c][3]));
            sum2 = add2(sum2, part);
        }
        const int width = WIDE ? 32 : team;
        const float2 halves = split(sum2);
        float sum = halves.x + halves.y;
        for (int o = width / 2; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        float mean = sum * inv_own;
        f32x2 shift = pair_of(-mean, -mean), dev2[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (t + c * span >= pieces) continue;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const f32x2 d = add2(v[c][i], shift);
                if constexpr (!WIDE) v[c][i] = d;
                dev2[i & 1] = fma2(d, d, dev2[i & 1]);
            }
        }
        const float2 devs = split(add2(dev2[0], dev2[1]));
        float dev = devs.x + devs.y;
        for (int o = width / 2; o; o >>= 1) dev += __shfl_xor_sync(0xFFFFFFFFu, dev, o);
        if constexpr (WIDE) {
            // two buffers: a warp that runs ahead writes the other one, and cannot reach this one
            // again before every warp has passed the next row's barrier
            if (lane == 0) {
                s_mean[buf][warp] = mean;
                s_dev[buf][warp] = dev;
            }
            __syncthreads();
            sum = 0.0f;
            for (int k = 0; k < nw; ++k) sum = __fmaf_rn(s_n[k], s_mean[buf][k], sum);
            mean = sum * inv_n;
            dev = 0.0f;
            for (int k = 0; k < nw; ++k) {
                const float m = s_mean[buf][k] - mean;
                dev = __fadd_rn(dev, __fmaf_rn(__fmul_rn(s_n[k], m), m, s_dev[buf][k]));
            }
            buf ^= 1;
            shift = pair_of(-mean, -mean);
        }
        const float rstd = 1.0f / sqrtf(__fmaf_rn(dev, inv_n, p.eps));
        const f32x2 scale = pair_of(rstd, rstd);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t + c * span;
            if (row >= p.M || k >= pieces) continue;
            const int64_t j = static_cast<int64_t>(k) * V;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const f32x2 d = WIDE ? add2(v[c][i], shift) : v[c][i];
                v[c][i] = fma2(mul2(d, scale), w[c][i], b[c][i]);
            }
            Piece<T, V> y;
            pack2(y, v[c]);
            if (p.y) y.store(p.y + row * p.ldy + j);
            if (p.quant.on) {
                uint8_t* dst = p.quant.q ? p.quant.q + row * p.N + j : nullptr;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    if (p.quant.fmt == FP8Q_E5M2) quant_bf16x8<FP8Q_E5M2>(s, y.raw, dst, amax2, nsat);
                    else quant_bf16x8<FP8Q_E4M3>(s, y.raw, dst, amax2, nsat);
                } else {
                    quant_piece<T, V>(p.quant, s, y, dst, amax, nsat);
                }
            }
        }
        if (row < p.M && t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
    if (p.quant.on) publish_quant(p.quant, max(amax, max16x2(amax2) << 16), nsat);
}

template <typename T, int V, int C, bool DROP, bool RES, bool WIDE>
cudaError_t launch_ring_as(const FwdParams<T>& p, int team, unsigned block, cudaStream_t stream) {
    // one wave: as many CTAs as run at a time (the answer is kept per CTA size)
    static std::atomic<int> per_sm[17];
    const auto kern = ln_fwd_ring_kernel<T, V, C, DROP, RES, WIDE>;
    const size_t smem = size_t(kRing) * (RES ? 2 : 1) * C * block * 16;
    int n = per_sm[block / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, static_cast<int>(block), smem);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
        per_sm[block / 32].store(n, std::memory_order_relaxed);
    }
    const int64_t rows = WIDE ? 1 : 128 / team;
    const int64_t grid = std::min<int64_t>((p.M + rows - 1) / rows, int64_t(n) * sm_count());
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, p, team);
}

template <typename T, int V, int C, bool WIDE>
cudaError_t launch_ring(const FwdParams<T>& p, int team, unsigned block, cudaStream_t stream) {
    if (p.drop.on)
        return p.res ? launch_ring_as<T, V, C, true, true, WIDE>(p, team, block, stream)
                     : launch_ring_as<T, V, C, true, false, WIDE>(p, team, block, stream);
    return p.res ? launch_ring_as<T, V, C, false, true, WIDE>(p, team, block, stream)
                 : launch_ring_as<T, V, C, false, false, WIDE>(p, team, block, stream);
}

template <typename T, int V, int C, bool WIDE>
cudaError_t launch_rows(const FwdParams<T>& p, int team, unsigned grid, unsigned block, cudaStream_t stream) {
    return p.drop.on ? launch_pdl(ln_fwd_rows_kernel<T, V, C, true, WIDE>, dim3(grid), dim3(block), 0, stream, p, team)
                     : launch_pdl(ln_fwd_rows_kernel<T, V, C, false, WIDE>, dim3(grid), dim3(block), 0, stream, p, team);
}

// The register kernels, where the row fits one; cudaErrorNotSupported where it does not.
template <typename T, int V>
cudaError_t launch_fwd_rows(const FwdParams<T>& p, cudaStream_t stream) {
    constexpr int kWide = V == 1 ? 8 : 4;  // pieces of a thread of a CTA's row
    const int64_t pieces = p.N / V;
    if constexpr (V > 1) {
        constexpr int kMost = 16 / V;
        if (pieces > 32 * 8 && pieces <= 512 * kMost)
            return launch_ring<T, V, kMost, true>(p, 0, static_cast<unsigned>((pieces + 32 * kMost - 1) / (32 * kMost)) * 32, stream);
        int team = 1;
        while (team < 32 && team < pieces) team *= 2;
        switch ((pieces + team - 1) / team) {
            case 1: return launch_ring<T, V, 1, false>(p, team, 128, stream);
            case 2: return launch_ring<T, V, 2, false>(p, team, 128, stream);
            case 3: return launch_ring<T, V, 3, false>(p, team, 128, stream);
            case 4: return launch_ring<T, V, 4, false>(p, team, 128, stream);
            case 5: return launch_ring<T, V, 5, false>(p, team, 128, stream);
            case 6: return launch_ring<T, V, 6, false>(p, team, 128, stream);
            case 7: return launch_ring<T, V, 7, false>(p, team, 128, stream);
            case 8: return launch_ring<T, V, 8, false>(p, team, 128, stream);
            default: break;
        }
    }
    if (pieces > 1024 * kWide) return cudaErrorNotSupported;
    if (pieces > 32 * 8) {
        const unsigned block = static_cast<unsigned>((pieces + 32 * kWide - 1) / (32 * kWide)) * 32;
        return launch_rows<T, V, kWide, true>(p, 0, static_cast<unsigned>(p.M), block, stream);
    }
    if constexpr (V == 1) {
    int team = 1;
    while (team < 32 && team < pieces) team *= 2;
    const unsigned grid = static_cast<unsigned>((p.M * team + 127) / 128);
    switch ((pieces + team - 1) / team) {
        case 1: return launch_rows<T, V, 1, false>(p, team, grid, 128, stream);
        case 2: return launch_rows<T, V, 2, false>(p, team, grid, 128, stream);
        case 3: return launch_rows<T, V, 3, false>(p, team, grid, 128, stream);
        case 4: return launch_rows<T, V, 4, false>(p, team, grid, 128, stream);
        case 5: return launch_rows<T, V, 5, false>(p, team, grid, 128, stream);
        case 6: return launch_rows<T, V, 6, false>(p, team, grid, 128, stream);
        case 7: return launch_rows<T, V, 7, false>(p, team, grid, 128, stream);
        default: return launch_rows<T, V, 8, false>(p, team, grid, 128, stream);
    }
    }
    return cudaErrorNotSupported;
}

template <typename T>
int launch_fwd(const fp8q_layer_norm_args& a, const Dropout& drop, const QuantOut& quant, cudaStream_t stream) {
    FwdParams<T> p;
    p.M = a.M;
    p.N = a.N;
    p.x = static_cast<const T*>(a.x);
    p.ldx = a.ldx;
    p.res = static_cast<const T*>(a.residual);
    p.ld_res = a.ld_residual;
    p.r_out = static_cast<T*>(a.r_out);
    p.ld_r = a.ld_r;
    p.w = Params<T>{a.weight, a.param_dtype == FP8Q_FP32, 1.0f};
    p.b = Params<T>{a.bias, a.param_dtype == FP8Q_FP32, 0.0f};
    p.eps = a.eps;
    p.y = static_cast<T*>(a.y);
    p.ldy = a.ldy;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.drop = drop;
    p.quant = quant;
    constexpr int V = 16 / sizeof(T);
    const bool pieces = a.N % V == 0 && rows16(a.x, a.ldx, sizeof(T)) && rows16(a.residual, a.ld_residual, sizeof(T)) &&
                        rows16(a.r_out, a.ld_r, sizeof(T)) && rows16(a.y, a.ldy, sizeof(T)) && aligned16(a.weight) &&
                        aligned16(a.bias) && aligned_to(a.q_out, V);
    cudaError_t e = pieces ? launch_fwd_rows<T, V>(p, stream) : launch_fwd_rows<T, 1>(p, stream);
    if (e == cudaErrorNotSupported) {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, int64_t(sm_count()) * 8));
        e = launch_pdl(ln_fwd_loop_kernel<T>, dim3(grid), dim3(256), 0, stream, p);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return FP8Q_OK;
}

}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" int layer_norm_fwd(const fp8q_layer_norm_args* args, cudaStream_t stream) {
    if (!args) return FP8Q_ERR_NULL;
    const fp8q_layer_norm_args& a = *args;
    if (!is_dtype(a.dtype) || (a.param_dtype != FP8Q_FP32 && a.param_dtype != a.dtype)) return FP8Q_ERR_UNSUPPORTED;
    if (a.flags & ~static_cast<unsigned>(FP8Q_ACCUMULATE)) return FP8Q_ERR_UNSUPPORTED;
    if (a.M < 0 || a.N < 1 || a.M > FP8Q_NORM_MAX || a.N > FP8Q_NORM_MAX) return FP8Q_ERR_SHAPE;
    QuantOut quant = {a.scale, static_cast<uint8_t*>(a.q_out), a.amax_out, a.sat_count, a.fmt,
                      a.q_out || a.amax_out || a.sat_count};
    if (quant.on) {
        if (a.fmt != FP8Q_E4M3 && a.fmt != FP8Q_E5M2) return FP8Q_ERR_UNSUPPORTED;
        if (!a.scale) return FP8Q_ERR_NULL;
    }
    Dropout drop;
    if (!make_dropout(a.p, a.rng, &drop)) return FP8Q_ERR_SHAPE;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps)) return FP8Q_ERR_SHAPE;
    if (a.M > 0 && (!a.x || (!a.y && !a.q_out) || (drop.on && !a.rng))) return FP8Q_ERR_NULL;
    const int64_t lds[4] = {a.ldx, a.residual ? a.ld_residual : a.N, a.r_out ? a.ld_r : a.N, a.y ? a.ldy : a.N};
    for (int64_t ld : lds)
        if (ld < a.N) return FP8Q_ERR_SHAPE;
    const size_t es = dtype_size(a.dtype), ps = dtype_size(a.param_dtype);
    if (!aligned_to(a.x, es) || !aligned_to(a.residual, es) || !aligned_to(a.r_out, es) || !aligned_to(a.y, es) ||
        !aligned_to(a.weight, ps) || !aligned_to(a.bias, ps) || !aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4) ||
        !aligned_to(a.rng, 8) || !aligned_to(a.scale, 4) || !aligned_to(a.amax_out, 4) || !aligned_to(a.sat_count, 8))
        return FP8Q_ERR_ALIGN;
    if (!device_is_sm103()) return FP8Q_ERR_UNSUPPORTED;

    if (!(a.flags & FP8Q_ACCUMULATE) && (a.amax_out || a.sat_count)) {
        if (launch_pdl(clear_quant_kernel, dim3(1), dim3(1), 0, stream, a.amax_out, a.sat_count) != cudaSuccess) {
            (void)cudaGetLastError();
            return FP8Q_ERR_CUDA;
        }
    }
    if (a.M == 0) return FP8Q_OK;
    switch (a.dtype) {
        case FP8Q_BF16: return launch_fwd<__nv_bfloat16>(a, drop, quant, stream);
        case FP8Q_FP16: return launch_fwd<__half>(a, drop, quant, stream);
        default: return launch_fwd<float>(a, drop, quant, stream);
    }
}
