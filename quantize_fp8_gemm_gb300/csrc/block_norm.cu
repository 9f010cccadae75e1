// block_norm.cu -- block_norm_fwd and block_norm_bwd: the norm after a block, its gate, the
// scaled residual and the norm before the next block (with its FP8 cast) in one pass, and
// their gradient.
//
//     xhat = post ? x rstd_post : x              rstd_post = 1 / sqrt(sum x^2 / N + eps)
//     r    = T(alpha residual + gate_i (xhat wp))
//     y    = T(r rstd w)                         rstd = 1 / sqrt(sum r^2 / N + eps)
//     q    = FP8(float32(y s)), max |y|, #{|y s| > max}
//
//     rhat = r rstd, g = dy w;  dr = dr_in + rstd (g - rhat sum(g rhat) / N)
//     dresidual = T(alpha dr);  dalpha = sum dr residual
//     e_i  = sum_j dr wp xhat;  dgate_i = e_i;  dx = T(gate_i rstd_post (dr wp - xhat e_i / N))
//     dw   = sum_i dy rhat;     dwp = sum_i gate_i dr xhat
//
// The norm before the next block is that of the stored r, so its gradient is that of what
// was computed.  Column sums and dalpha go through float32 partial rows in the caller's
// workspace, which a second kernel adds in a fixed order.  The one-pass kernels are in
// block_norm.cuh, those for any width here.
#include "block_norm.cuh"

#include <algorithm>
#include <cmath>

namespace fp8q {

// in block_norm_*.cu
#define FP8Q_BN_EXTERN(T, SHIFT)                                                              \
    extern template cudaError_t launch_bn_fwd<T, SHIFT>(const BnFwd<T>&, cudaStream_t);       \
    extern template cudaError_t launch_bn_bwd<T, false, SHIFT>(const BnBwd<T>&, int, int*, cudaStream_t); \
    extern template cudaError_t launch_bn_bwd<T, true, SHIFT>(const BnBwd<T>&, int, int*, cudaStream_t);
FP8Q_BN_EXTERN(__nv_bfloat16, false)
FP8Q_BN_EXTERN(__nv_bfloat16, true)
FP8Q_BN_EXTERN(__half, false)
FP8Q_BN_EXTERN(__half, true)
FP8Q_BN_EXTERN(float, false)
FP8Q_BN_EXTERN(float, true)
#undef FP8Q_BN_EXTERN

namespace {

// Rows wider than the one-pass kernels take: one CTA a row, in passes over it (the later ones
// from L1 / L2).  The row is formed again in every pass and written in the last, element by
// element by the thread that read it, so an output may replace an input.  Far from any bound of the hardware (of
// the copy rate: forward bf16 4096 x 20001 542 us, 0.18, 1024 x 65536 638, 0.12; float32 688, 0.28, and 665, 0.24;
// backward, which comes here past 65536 two-byte or 32768 four-byte columns, bf16 1024 x 100000 3.2 ms, 0.06, float32
// 2.6 ms, 0.14); no counters were taken, the code loads single elements and keeps its column sums in memory.
template <typename T>
__device__ __forceinline__ float bn_stream(const BnFwd<T>& p, int64_t row, int64_t j, float rp, float gate, float alpha) {
    float v = __fmul_rn(__fmul_rn(__fmul_rn(to_f32(p.x[row * p.ldx + j]), rp), p.wp.at(j)), gate);
    if (p.res) v = __fmaf_rn(alpha, to_f32(p.res[row * p.ld_res + j]), v);
    return round_to<T>(v);
}

template <typename T>
__global__ void __launch_bounds__(512) bn_fwd_loop_kernel(const BnFwd<T> p) {
    __shared__ float s_sum[66];
    pdl_wait();
    const float inv_n = 1.0f / static_cast<float>(p.N);
    const float s = p.quant.on ? *p.quant.scale : 0.0f, alpha = p.alpha ? *p.alpha : 1.0f;
    const float fmax = fp8_max_value(p.quant.fmt);
    uint32_t amax = 0, nsat = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const float gate = p.gate ? p.gate[row] : 1.0f;
        float rp = 1.0f, rstd = 1.0f;
        if (p.post) {
            float sum = 0.0f;
            for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x) {
                const float v = to_f32(p.x[row * p.ldx + j]);
                sum = __fmaf_rn(v, v, sum);
            }
            rp = 1.0f / sqrtf(__fmaf_rn(block_sum2(sum, 0.0f, s_sum).x, inv_n, p.eps));
        }
        if (p.pre) {
            float sum = 0.0f;
            for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x) {
                const float v = bn_stream(p, row, j, rp, gate, alpha);
                sum = __fmaf_rn(v, v, sum);
            }
            rstd = 1.0f / sqrtf(__fmaf_rn(block_sum2(sum, 0.0f, s_sum).x, inv_n, p.eps));
        }
        for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x) {
            const float r = bn_stream(p, row, j, rp, gate, alpha);
            if (p.r_out) p.r_out[row * p.ld_r + j] = from_f32<T>(r);
            if (!p.pre) continue;
            const T y = from_f32<T>(__fmul_rn(__fmul_rn(r, rstd), p.w.at(j)));
            if (p.y) p.y[row * p.ldy + j] = y;
            if (p.quant.on) {
                const float yf = to_f32(y), v = __fmul_rn(yf, s);
                amax = max(amax, __float_as_uint(fabsf(yf)));
                nsat += fabsf(v) > fmax;
                if (p.quant.q) p.quant.q[row * p.N + j] = static_cast<uint8_t>(cast_pair(v, 0.0f, p.quant.fmt));
            }
        }
        if (threadIdx.x == 0) {
            if (p.rstd_post && p.post) p.rstd_post[row] = rp;
            if (p.rstd && p.pre) p.rstd[row] = rstd;
        }
    }
    pdl_launch_dependents();
    finish_quant(p, amax, nsat);
}

// The stream's gradient at one element, `along` = sum(g rhat) / N.
template <typename T>
__device__ __forceinline__ float bn_dr(const BnBwd<T>& p, int64_t row, int64_t j, float rstd, float along, float& dy, float& rhat) {
    float d = p.dr ? to_f32(p.dr[row * p.ld_dr + j]) : 0.0f;
    if (p.dy) {
        dy = to_f32(p.dy[row * p.ld_dy + j]);
        rhat = __fmul_rn(to_f32(p.r[row * p.ld_r + j]), rstd);
        d = __fmaf_rn(__fmaf_rn(rhat, -along, __fmul_rn(dy, p.w.at(j))), rstd, d);
    }
    return d;
}

// A CTA adds its rows' terms to its own partial row in memory.
template <typename T>
__global__ void __launch_bounds__(512) bn_bwd_loop_kernel(const BnBwd<T> p) {
    __shared__ float s_sum[66];
    pdl_wait();
    const float inv_n = 1.0f / static_cast<float>(p.N), alpha = p.alpha ? *p.alpha : 1.0f;
    float* const part = p.part ? p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.N : nullptr;
    float dalpha = 0.0f;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const float gate = p.gate ? p.gate[row] : 1.0f, rp = p.rstd_post ? p.rstd_post[row] : 1.0f;
        const float rstd = p.dy ? p.rstd[row] : 0.0f;
        float along = 0.0f, dy = 0.0f, rhat = 0.0f, e = 0.0f;
        if (p.dy) {
            float sum = 0.0f;
            for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x)
                sum = __fmaf_rn(to_f32(p.dy[row * p.ld_dy + j]) * p.w.at(j), __fmul_rn(to_f32(p.r[row * p.ld_r + j]), rstd), sum);
            along = block_sum2(sum, 0.0f, s_sum).x * inv_n;
        }
        if (p.x) {
            float sum = 0.0f;
            for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x)
                sum = __fmaf_rn(bn_dr(p, row, j, rstd, along, dy, rhat) * p.wp.at(j), __fmul_rn(to_f32(p.x[row * p.ldx + j]), rp), sum);
            e = block_sum2(sum, 0.0f, s_sum).x;
            if (p.dgate && threadIdx.x == 0) p.dgate[row] = e;
        }
        for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x) {
            const float d = bn_dr(p, row, j, rstd, along, dy, rhat);
            if (p.res) dalpha = __fmaf_rn(d, to_f32(p.res[row * p.ld_res + j]), dalpha);
            const float xhat = p.x ? __fmul_rn(to_f32(p.x[row * p.ldx + j]), rp) : 0.0f;
            if (part) {
                part[j] = first ? dy * rhat : __fmaf_rn(dy, rhat, part[j]);
                part[p.N + j] = first ? d * gate * xhat : __fmaf_rn(d * gate, xhat, part[p.N + j]);
            }
            if (p.dres) p.dres[row * p.ld_dres + j] = from_f32<T>(d * alpha);
            if (p.dx) {
                float f = d * p.wp.at(j);
                if (p.post) f = __fmaf_rn(xhat, -e * inv_n, f) * rp;
                p.dx[row * p.ld_dx + j] = from_f32<T>(f * gate);
            }
        }
        first = false;
    }
    dalpha = block_sum2(dalpha, 0.0f, s_sum).x;
    if (part && threadIdx.x == 0) p.part[static_cast<int64_t>(p.parts) * 2 * p.N + blockIdx.x] = dalpha;
    pdl_launch_dependents();
}

// dweight, dpost_weight and dalpha = the partial rows' sums in a fixed order.  A block takes 32
// columns of [2][N] (the last block dalpha); warp k of its 16 adds parts k, k + 16, ..., then the
// warps' sums are added in order.
constexpr int kBnReduceWarps = 16;
__global__ void __launch_bounds__(kBnReduceWarps * 32)
bn_bwd_reduce_kernel(const float* part, int parts, int64_t N, float* dweight, float* dpost, float* dalpha, bool accumulate) {
    __shared__ float s[kBnReduceWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool cell = static_cast<int64_t>(blockIdx.x) * 32 >= 2 * N;
    const int64_t j = cell ? 2 * N : static_cast<int64_t>(blockIdx.x) * 32 + lane;
    pdl_wait();
    float sum = 0.0f;
    if (cell) {
        for (int k = threadIdx.x; k < parts; k += blockDim.x) sum += part[static_cast<int64_t>(parts) * 2 * N + k];
        sum = team_sum<false>(sum, 32);
    } else if (j < 2 * N) {
        constexpr int kAtOnce = 10;
        for (int k0 = warp; k0 < parts; k0 += kAtOnce * kBnReduceWarps) {
            float v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int k = k0 + u * kBnReduceWarps;
                v[u] = k < parts ? part[static_cast<int64_t>(k) * 2 * N + j] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) sum += v[u];
        }
    }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kBnReduceWarps; ++k) sum += s[k][lane];
        float* out = cell ? (lane == 0 ? dalpha : nullptr) : j < N ? (dweight ? dweight + j : nullptr)
                   : j < 2 * N && dpost ? dpost + (j - N) : nullptr;
        if (out) *out = accumulate ? *out + sum : sum;
    }
    pdl_launch_dependents();
}

// Most partial rows of a call: CTAs of the row kernels that run at a time.
int bn_parts(int64_t M) { return static_cast<int>(std::min<int64_t>(M, std::min(1024, 4 * sm_count()))); }

template <typename T>
int run_bn_fwd(const fp8q_block_norm_args& a, const QuantOut& quant, cudaStream_t stream) {
    BnFwd<T> p = {};
    p.M = a.M;
    p.N = a.N;
    p.x = static_cast<const T*>(a.x);
    p.ldx = a.ldx;
    p.res = static_cast<const T*>(a.residual);
    p.ld_res = a.ld_residual;
    p.r_out = static_cast<T*>(a.r_out);
    p.ld_r = a.ld_r;
    p.y = static_cast<T*>(a.y);
    p.ldy = a.ldy;
    p.w = Params<T>{a.weight, a.param_dtype == FP8Q_FP32, 1.0f, aligned16(a.weight)};
    p.wp = Params<T>{a.post_weight, a.param_dtype == FP8Q_FP32, 1.0f, aligned16(a.post_weight)};
    p.gate = a.gate;
    p.alpha = a.alpha;
    p.rstd = a.rstd;
    p.rstd_post = a.rstd_post;
    p.eps = a.eps;
    p.post = a.post_norm != 0;
    p.pre = a.y || quant.on || a.rstd;
    p.quant = quant;
    p.alone = a.M == 1 && !(a.flags & FP8Q_ACCUMULATE);  // (one row is one CTA)
    constexpr int V = 16 / sizeof(T);
    const bool grid16 = a.N % V == 0 && rows16(a.x, a.ldx, sizeof(T)) && rows16(a.residual, a.ld_residual, sizeof(T)) &&
                        rows16(a.r_out, a.ld_r, sizeof(T)) && rows16(a.y, a.ldy, sizeof(T)) && aligned16(a.weight) &&
                        aligned16(a.post_weight) && aligned_to(a.q_out, V);
    cudaError_t e = grid16 ? launch_bn_fwd<T, false>(p, stream) : launch_bn_fwd<T, true>(p, stream);
    if (e == cudaErrorNotSupported)
        e = launch_pdl(bn_fwd_loop_kernel<T>, dim3(static_cast<unsigned>(std::min<int64_t>(a.M, int64_t(sm_count()) * 4))),
                       dim3(512), 0, stream, p);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return FP8Q_OK;
}

template <typename T>
int run_bn_bwd(const fp8q_block_norm_bwd_args& a, cudaStream_t stream) {
    BnBwd<T> p = {};
    p.M = a.M;
    p.N = a.N;
    p.dy = static_cast<const T*>(a.dy);
    p.ld_dy = a.ld_dy;
    p.r = static_cast<const T*>(a.dy ? a.r : nullptr);
    p.ld_r = a.ld_r;
    p.dr = static_cast<const T*>(a.dr);
    p.ld_dr = a.ld_dr;
    const bool block = a.dx || a.dpost_weight || a.dgate;
    p.x = block ? static_cast<const T*>(a.x) : nullptr;
    p.ldx = a.ldx;
    p.res = a.dalpha ? static_cast<const T*>(a.residual) : nullptr;
    p.ld_res = a.ld_residual;
    p.dres = static_cast<T*>(a.dresidual);
    p.ld_dres = a.ld_dresidual;
    p.dx = static_cast<T*>(a.dx);
    p.ld_dx = a.ld_dx;
    p.w = Params<T>{a.weight, a.param_dtype == FP8Q_FP32, 1.0f, aligned16(a.weight)};
    p.wp = Params<T>{a.post_weight, a.param_dtype == FP8Q_FP32, 1.0f, aligned16(a.post_weight)};
    p.gate = a.gate;
    p.alpha = a.alpha;
    p.rstd = a.rstd;
    p.post = a.post_norm != 0;
    p.rstd_post = block && p.post ? a.rstd_post : nullptr;
    p.dgate = a.dgate;
    const bool sums = a.dweight || a.dpost_weight || a.dalpha;
    p.part = sums ? static_cast<float*>(a.workspace) : nullptr;
    constexpr int V = 16 / sizeof(T);
    const bool grid16 = a.N % V == 0 && rows16(p.dy, a.ld_dy, sizeof(T)) && rows16(p.r, a.ld_r, sizeof(T)) &&
                        rows16(p.dr, a.ld_dr, sizeof(T)) && rows16(p.x, a.ldx, sizeof(T)) &&
                        rows16(p.res, a.ld_residual, sizeof(T)) && rows16(p.dres, a.ld_dresidual, sizeof(T)) &&
                        rows16(p.dx, a.ld_dx, sizeof(T)) && aligned16(a.weight) && aligned16(a.post_weight);
    const int most = bn_parts(a.M);
    int parts = most;
    cudaError_t e;
    if (p.res) e = grid16 ? launch_bn_bwd<T, true, false>(p, most, &parts, stream) : launch_bn_bwd<T, true, true>(p, most, &parts, stream);
    else e = grid16 ? launch_bn_bwd<T, false, false>(p, most, &parts, stream) : launch_bn_bwd<T, false, true>(p, most, &parts, stream);
    if (e == cudaErrorNotSupported) {
        p.parts = parts = most;
        e = launch_pdl(bn_bwd_loop_kernel<T>, dim3(static_cast<unsigned>(parts)), dim3(512), 0, stream, p);
    }
    if (sums && e == cudaSuccess)
        e = launch_pdl(bn_bwd_reduce_kernel, dim3(static_cast<unsigned>((2 * a.N + 31) / 32 + (a.dalpha ? 1 : 0))),
                       dim3(kBnReduceWarps * 32), 0, stream, static_cast<const float*>(p.part), parts, a.N, a.dweight,
                       a.dpost_weight, a.dalpha, (a.flags & FP8Q_ACCUMULATE) != 0);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return FP8Q_OK;
}

bool ld_ok(const void* p, int64_t ld, int64_t N) { return p == nullptr || ld >= N; }

}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" int block_norm_fwd(const fp8q_block_norm_args* args, cudaStream_t stream) {
    if (!args) return FP8Q_ERR_NULL;
    const fp8q_block_norm_args& a = *args;
    if (!is_dtype(a.dtype) || (a.param_dtype != FP8Q_FP32 && a.param_dtype != a.dtype)) return FP8Q_ERR_UNSUPPORTED;
    if (a.flags & ~static_cast<unsigned>(FP8Q_ACCUMULATE)) return FP8Q_ERR_UNSUPPORTED;
    if (a.M < 0 || a.N < 1 || a.M > FP8Q_NORM_MAX || a.N > FP8Q_NORM_MAX) return FP8Q_ERR_SHAPE;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps)) return FP8Q_ERR_SHAPE;
    const QuantOut quant = {a.scale, static_cast<uint8_t*>(a.q_out), a.amax_out, a.sat_count, a.fmt,
                            a.q_out || a.amax_out || a.sat_count};
    if (quant.on) {
        if (a.fmt != FP8Q_E4M3 && a.fmt != FP8Q_E5M2) return FP8Q_ERR_UNSUPPORTED;
        if (!a.scale) return FP8Q_ERR_NULL;
    }
    if (a.M > 0 && (!a.x || (!a.y && !a.q_out && !a.r_out))) return FP8Q_ERR_NULL;
    if (!ld_ok(a.x, a.ldx, a.N) || !ld_ok(a.residual, a.ld_residual, a.N) || !ld_ok(a.r_out, a.ld_r, a.N) ||
        !ld_ok(a.y, a.ldy, a.N))
        return FP8Q_ERR_SHAPE;
    const size_t es = dtype_size(a.dtype), ps = dtype_size(a.param_dtype);
    if (!aligned_to(a.x, es) || !aligned_to(a.residual, es) || !aligned_to(a.r_out, es) || !aligned_to(a.y, es) ||
        !aligned_to(a.weight, ps) || !aligned_to(a.post_weight, ps) || !aligned_to(a.gate, 4) || !aligned_to(a.alpha, 4) ||
        !aligned_to(a.rstd, 4) || !aligned_to(a.rstd_post, 4) || !aligned_to(a.scale, 4) || !aligned_to(a.amax_out, 4) ||
        !aligned_to(a.sat_count, 8))
        return FP8Q_ERR_ALIGN;
    if (!device_is_sm103()) return FP8Q_ERR_UNSUPPORTED;
    if (!(a.flags & FP8Q_ACCUMULATE) && (a.amax_out || a.sat_count) && a.M != 1) {
        if (launch_pdl(clear_quant_kernel, dim3(1), dim3(1), 0, stream, a.amax_out, a.sat_count) != cudaSuccess) {
            (void)cudaGetLastError();
            return FP8Q_ERR_CUDA;
        }
    }
    if (a.M == 0) return FP8Q_OK;
    switch (a.dtype) {
        case FP8Q_BF16: return run_bn_fwd<__nv_bfloat16>(a, quant, stream);
        case FP8Q_FP16: return run_bn_fwd<__half>(a, quant, stream);
        default: return run_bn_fwd<float>(a, quant, stream);
    }
}

extern "C" size_t block_norm_bwd_workspace_bytes(int64_t M, int64_t N) {
    if (M < 1 || N < 1 || M > FP8Q_NORM_MAX || N > FP8Q_NORM_MAX) return 0;
    const size_t parts = static_cast<size_t>(bn_parts(M));
    return (parts * (2 * static_cast<size_t>(N) + 1) * sizeof(float) + 15) / 16 * 16;
}

extern "C" int block_norm_bwd(const fp8q_block_norm_bwd_args* args, cudaStream_t stream) {
    if (!args) return FP8Q_ERR_NULL;
    const fp8q_block_norm_bwd_args& a = *args;
    if (!is_dtype(a.dtype) || (a.param_dtype != FP8Q_FP32 && a.param_dtype != a.dtype)) return FP8Q_ERR_UNSUPPORTED;
    if (a.flags & ~static_cast<unsigned>(FP8Q_ACCUMULATE)) return FP8Q_ERR_UNSUPPORTED;
    if (a.M < 0 || a.N < 1 || a.M > FP8Q_NORM_MAX || a.N > FP8Q_NORM_MAX) return FP8Q_ERR_SHAPE;
    const bool block = a.dx || a.dpost_weight || a.dgate, sums = a.dweight || a.dpost_weight || a.dalpha;
    if (a.M > 0) {
        if (!a.dy && !a.dr) return FP8Q_ERR_NULL;
        if (a.dy ? !a.r || !a.rstd : a.dweight != nullptr) return FP8Q_ERR_NULL;
        if (block && (!a.x || (a.post_norm && !a.rstd_post))) return FP8Q_ERR_NULL;
        if (a.dalpha && !a.residual) return FP8Q_ERR_NULL;
        if (!a.dresidual && !block && !sums) return FP8Q_ERR_NULL;
        if (sums && !a.workspace) return FP8Q_ERR_NULL;
    }
    if (!ld_ok(a.dy, a.ld_dy, a.N) || !ld_ok(a.r, a.ld_r, a.N) || !ld_ok(a.dr, a.ld_dr, a.N) || !ld_ok(a.x, a.ldx, a.N) ||
        !ld_ok(a.residual, a.ld_residual, a.N) || !ld_ok(a.dresidual, a.ld_dresidual, a.N) || !ld_ok(a.dx, a.ld_dx, a.N))
        return FP8Q_ERR_SHAPE;
    const size_t es = dtype_size(a.dtype), ps = dtype_size(a.param_dtype);
    if (!aligned_to(a.dy, es) || !aligned_to(a.r, es) || !aligned_to(a.dr, es) || !aligned_to(a.x, es) ||
        !aligned_to(a.residual, es) || !aligned_to(a.dresidual, es) || !aligned_to(a.dx, es) ||
        !aligned_to(a.weight, ps) || !aligned_to(a.post_weight, ps) || !aligned_to(a.gate, 4) || !aligned_to(a.alpha, 4) ||
        !aligned_to(a.rstd, 4) || !aligned_to(a.rstd_post, 4) || !aligned_to(a.dweight, 4) ||
        !aligned_to(a.dpost_weight, 4) || !aligned_to(a.dgate, 4) || !aligned_to(a.dalpha, 4) || !aligned_to(a.workspace, 16))
        return FP8Q_ERR_ALIGN;
    if (!device_is_sm103()) return FP8Q_ERR_UNSUPPORTED;
    if (a.M > 0 && sums && a.workspace_bytes < block_norm_bwd_workspace_bytes(a.M, a.N)) return FP8Q_ERR_SHAPE;
    if (a.M == 0) {  // no rows: the sums are zero, and nothing is added to what accumulates
        if (a.flags & FP8Q_ACCUMULATE) return FP8Q_OK;
        if (a.dweight && cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.N, stream) != cudaSuccess) return FP8Q_ERR_CUDA;
        if (a.dpost_weight && cudaMemsetAsync(a.dpost_weight, 0, sizeof(float) * a.N, stream) != cudaSuccess) return FP8Q_ERR_CUDA;
        if (a.dalpha && cudaMemsetAsync(a.dalpha, 0, sizeof(float), stream) != cudaSuccess) return FP8Q_ERR_CUDA;
        return FP8Q_OK;
    }
    switch (a.dtype) {
        case FP8Q_BF16: return run_bn_bwd<__nv_bfloat16>(a, stream);
        case FP8Q_FP16: return run_bn_bwd<__half>(a, stream);
        default: return run_bn_bwd<float>(a, stream);
    }
}
