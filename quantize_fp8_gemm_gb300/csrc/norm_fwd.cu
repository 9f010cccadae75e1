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
// Statistics are float32 sums: the mean's, then the squared deviations' from it (not
// of squares), so a mean far above the deviation costs the variance no digits beyond
// the mean's own rounding.  The kernels are in norm_fwd.cuh, the one for
// any width here.
#include "norm_fwd.cuh"

#include <algorithm>
#include <cmath>

namespace fp8q {

__global__ void clear_quant_kernel(float* amax, unsigned long long* sat) {
    pdl_launch_dependents();
    pdl_wait();
    if (amax) *amax = 0.0f;
    if (sat) *sat = 0ull;
}

// in norm_fwd_*.cu
extern template cudaError_t launch_fwd_ring<__nv_bfloat16, false>(const FwdParams<__nv_bfloat16>&, cudaStream_t);
extern template cudaError_t launch_fwd_ring<__nv_bfloat16, true>(const FwdParams<__nv_bfloat16>&, cudaStream_t);
extern template cudaError_t launch_fwd_ring<__half, false>(const FwdParams<__half>&, cudaStream_t);
extern template cudaError_t launch_fwd_ring<__half, true>(const FwdParams<__half>&, cudaStream_t);
extern template cudaError_t launch_fwd_ring<float, false>(const FwdParams<float>&, cudaStream_t);
extern template cudaError_t launch_fwd_ring<float, true>(const FwdParams<float>&, cudaStream_t);

namespace {

// Wider than the one-pass kernels' 16384 columns: one CTA per row, three passes over the row (the second and third
// from L1 / L2), each thread taking quads of columns (one generator block).
// The row is formed again from its inputs in every pass and r_out is written
// in the last, so r_out and y may replace an input.
template <typename T>
__device__ __forceinline__ void row_quad(const FwdParams<T>& p, int64_t row, int64_t quad, float (&r)[4]) {
    const int64_t j0 = quad * 4;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (p.drop.on) w = Philox(p.drop.rng).at(static_cast<uint32_t>(quad), static_cast<uint32_t>(row));
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
    p.w = Params<T>{a.weight, a.param_dtype == FP8Q_FP32, 1.0f, aligned16(a.weight)};
    p.b = Params<T>{a.bias, a.param_dtype == FP8Q_FP32, 0.0f, aligned16(a.bias)};
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
    cudaError_t e = pieces ? launch_fwd_ring<T, false>(p, stream) : launch_fwd_ring<T, true>(p, stream);
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
