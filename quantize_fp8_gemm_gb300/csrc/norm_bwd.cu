// norm_bwd.cu -- layer_norm_bwd: the gradient of layer_norm_fwd.
//
// With xhat = (r - mean) * rstd and g = dy * w (per row, N columns):
//     dr      = rstd * (g - sum(g) / N - xhat * sum(g * xhat) / N) + dresidual
//     dx      = T(dr)                       gradient of r, and of the residual
//     dbranch = keep ? T(float32(dr * inv)) : 0       gradient of the branch x
//     dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy
// The column sums go through float32 partial rows in the caller's workspace,
// which a second kernel adds in a fixed order: no atomics, so the same call
// gives the same bits.
#include "norm_bwd.cuh"

#include <algorithm>

namespace fp8q {

// in norm_bwd_*.cu
extern template cudaError_t launch_bwd_ring<__nv_bfloat16, false>(BwdParams<__nv_bfloat16>&, cudaStream_t);
extern template cudaError_t launch_bwd_ring<__nv_bfloat16, true>(BwdParams<__nv_bfloat16>&, cudaStream_t);
extern template cudaError_t launch_bwd_ring<__half, false>(BwdParams<__half>&, cudaStream_t);
extern template cudaError_t launch_bwd_ring<__half, true>(BwdParams<__half>&, cudaStream_t);
extern template cudaError_t launch_bwd_ring<float, false>(BwdParams<float>&, cudaStream_t);
extern template cudaError_t launch_bwd_ring<float, true>(BwdParams<float>&, cudaStream_t);

namespace {

// Wider than the one-pass kernels' 16384 columns: one CTA per row, two passes over it.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_loop_kernel(const BwdParams<T> p) {
    __shared__ float s_sum[66];
    pdl_wait();
    const int64_t quads = (p.N + 3) / 4;
    const float inv_n = 1.0f / static_cast<float>(p.N);
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const T* dy = p.dy + row * p.ld_dy;
        const T* r = p.r + row * p.ld_r;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float c1 = 0.0f, c2 = 0.0f;
        for (int64_t j = threadIdx.x; j < p.N; j += blockDim.x) {
            const float g = to_f32(dy[j]) * p.w.at(j);
            c1 += g;
            c2 += g * ((to_f32(r[j]) - mean) * rstd);
        }
        const float2 c = block_sum2(c1, c2, s_sum);
        c1 = c.x * inv_n;
        c2 = c.y * inv_n;
        for (int64_t q = threadIdx.x; q < quads; q += blockDim.x) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (p.dbranch && p.drop.on)
                w = Philox(p.drop.rng).at(static_cast<uint32_t>(q), static_cast<uint32_t>(row));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t j = q * 4 + i;
                if (j >= p.N) continue;
                const float xhat = (to_f32(r[j]) - mean) * rstd;
                float d = rstd * (to_f32(dy[j]) * p.w.at(j) - c1 - xhat * c2);
                if (p.dres) d += to_f32(p.dres[row * p.ld_dres + j]);
                p.dx[row * p.ld_dx + j] = from_f32<T>(d);
                if (p.dbranch) p.dbranch[row * p.ld_db + j] = from_f32<T>(p.drop.on ? dropped(d, word_of(w, i), p.drop) : d);
            }
        }
    }
    pdl_launch_dependents();
}

// Column sums of rows part, part + parts, ...: a thread a column.  Runs before
// the row kernel, whose dx may replace dy or r.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_cols_kernel(const BwdParams<T> p) {
    pdl_wait();
    const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (j < p.N) {
        float dw = 0.0f, db = 0.0f;
        for (int64_t row = blockIdx.y; row < p.M; row += p.parts) {
            const float d = to_f32(p.dy[row * p.ld_dy + j]);
            dw += d * ((to_f32(p.r[row * p.ld_r + j]) - p.mean[row]) * p.rstd[row]);
            db += d;
        }
        float* part = p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.N;
        part[j] = dw;
        part[p.N + j] = db;
    }
    pdl_launch_dependents();
}

// dweight / dbias = the partial rows' sums in a fixed order.  A block takes 32
// columns; warp k of its 16 adds parts k, k + 16, ..., then the warps' sums are
// added by a tree of fixed shape.
constexpr int kReduceWarps = 16;
__global__ void __launch_bounds__(kReduceWarps * 32) ln_bwd_reduce_kernel(const float* part, int parts, int64_t N,
                                                                          float* dweight, float* dbias, bool accumulate) {
    __shared__ float s[kReduceWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // column of [2][N]
    pdl_wait();
    float sum = 0.0f;
    if (j < 2 * N) {
        // ten loads in flight: 160 parts a round (152 CTAs write one each)
        constexpr int kAtOnce = 10;
        for (int k0 = warp; k0 < parts; k0 += kAtOnce * kReduceWarps) {
            float v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int k = k0 + u * kReduceWarps;
                v[u] = k < parts ? part[static_cast<int64_t>(k) * 2 * N + j] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) sum += v[u];
        }
    }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp < kReduceWarps / 4 && j < 2 * N) {  // sixteen values of a column by fours
        sum = (s[4 * warp][lane] + s[4 * warp + 1][lane]) + (s[4 * warp + 2][lane] + s[4 * warp + 3][lane]);
        s[4 * warp][lane] = sum;
    }
    __syncthreads();
    if (warp == 0 && j < 2 * N) {
        sum = (s[0][lane] + s[4][lane]) + (s[8][lane] + s[12][lane]);
        float* out = j < N ? dweight : dbias;
        if (out) {
            out += j < N ? j : j - N;
            *out = accumulate ? *out + sum : sum;
        }
    }
    pdl_launch_dependents();
}

// Most partial rows of a call: CTAs of the row kernels that run at a time.
int parts_of(int64_t M, int64_t) { return static_cast<int>(std::min<int64_t>(M, std::min(1024, 4 * sm_count()))); }

template <typename T>
int launch_bwd(const fp8q_layer_norm_bwd_args& a, const Dropout& drop, cudaStream_t stream) {
    BwdParams<T> p;
    p.M = a.M;
    p.N = a.N;
    p.dy = static_cast<const T*>(a.dy);
    p.ld_dy = a.ld_dy;
    p.r = static_cast<const T*>(a.r);
    p.ld_r = a.ld_r;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.w = Params<T>{a.weight, a.param_dtype == FP8Q_FP32, 1.0f, aligned16(a.weight)};
    p.dres = static_cast<const T*>(a.dresidual);
    p.ld_dres = a.ld_dresidual;
    p.dx = static_cast<T*>(a.dx);
    p.ld_dx = a.ld_dx;
    p.dbranch = static_cast<T*>(a.dbranch);
    p.ld_db = a.ld_dbranch;
    p.drop = drop;
    p.part = static_cast<float*>(a.workspace);
    p.parts = parts_of(a.M, a.N);
    const bool cols = a.dweight || a.dbias;
    if (!cols) p.part = nullptr;
    p.dweight = a.dweight;
    p.dbias = a.dbias;
    p.accumulate = (a.flags & FP8Q_ACCUMULATE) != 0;
    bool reduce = cols;
    constexpr int V = 16 / sizeof(T);
    const bool pieces = a.N % V == 0 && rows16(a.dy, a.ld_dy, sizeof(T)) && rows16(a.r, a.ld_r, sizeof(T)) &&
                        rows16(a.dresidual, a.ld_dresidual, sizeof(T)) && rows16(a.dx, a.ld_dx, sizeof(T)) &&
                        rows16(a.dbranch, a.ld_dbranch, sizeof(T)) && aligned16(a.weight);
    cudaError_t e = pieces ? launch_bwd_ring<T, false>(p, stream) : launch_bwd_ring<T, true>(p, stream);
    if (e == cudaSuccess) reduce = cols && p.parts > 1;
    if (e == cudaErrorNotSupported) {
        e = cudaSuccess;
        if (cols)
            e = launch_pdl(ln_bwd_cols_kernel<T>, dim3(static_cast<unsigned>((a.N + 255) / 256), p.parts), dim3(256), 0,
                           stream, p);
        if (e == cudaSuccess)
            e = launch_pdl(ln_bwd_loop_kernel<T>,
                           dim3(static_cast<unsigned>(std::min<int64_t>(a.M, int64_t(sm_count()) * 8))), dim3(256), 0,
                           stream, p);
    }
    if (reduce && e == cudaSuccess)
        e = launch_pdl(ln_bwd_reduce_kernel, dim3(static_cast<unsigned>((2 * a.N + 31) / 32)), dim3(kReduceWarps * 32), 0, stream,
                       static_cast<const float*>(p.part), p.parts, a.N, a.dweight, a.dbias, p.accumulate);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return FP8Q_OK;
}

}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" size_t layer_norm_bwd_workspace_bytes(int64_t M, int64_t N) {
    if (M < 1 || N < 1 || M > FP8Q_NORM_MAX || N > FP8Q_NORM_MAX) return 0;
    return static_cast<size_t>(parts_of(M, N)) * 2 * static_cast<size_t>(N) * sizeof(float);
}

extern "C" int layer_norm_bwd(const fp8q_layer_norm_bwd_args* args, cudaStream_t stream) {
    if (!args) return FP8Q_ERR_NULL;
    const fp8q_layer_norm_bwd_args& a = *args;
    if (!is_dtype(a.dtype) || (a.param_dtype != FP8Q_FP32 && a.param_dtype != a.dtype)) return FP8Q_ERR_UNSUPPORTED;
    if (a.flags & ~static_cast<unsigned>(FP8Q_ACCUMULATE)) return FP8Q_ERR_UNSUPPORTED;
    if (a.M < 0 || a.N < 1 || a.M > FP8Q_NORM_MAX || a.N > FP8Q_NORM_MAX) return FP8Q_ERR_SHAPE;
    Dropout drop;
    if (!make_dropout(a.p, a.rng, &drop)) return FP8Q_ERR_SHAPE;
    const bool cols = a.dweight || a.dbias;
    if (a.M > 0 && (!a.dy || !a.r || !a.mean || !a.rstd || !a.dx || (a.dbranch && drop.on && !a.rng) ||
                    (cols && !a.workspace)))
        return FP8Q_ERR_NULL;
    const int64_t lds[5] = {a.ld_dy, a.ld_r, a.dresidual ? a.ld_dresidual : a.N, a.ld_dx, a.dbranch ? a.ld_dbranch : a.N};
    for (int64_t ld : lds)
        if (ld < a.N) return FP8Q_ERR_SHAPE;
    const size_t es = dtype_size(a.dtype);
    if (!aligned_to(a.dy, es) || !aligned_to(a.r, es) || !aligned_to(a.dresidual, es) || !aligned_to(a.dx, es) ||
        !aligned_to(a.dbranch, es) || !aligned_to(a.weight, dtype_size(a.param_dtype)) || !aligned_to(a.mean, 4) ||
        !aligned_to(a.rstd, 4) || !aligned_to(a.dweight, 4) || !aligned_to(a.dbias, 4) || !aligned_to(a.rng, 8) ||
        !aligned_to(a.workspace, 16))
        return FP8Q_ERR_ALIGN;
    if (a.M > 0 && cols && a.workspace_bytes < layer_norm_bwd_workspace_bytes(a.M, a.N)) return FP8Q_ERR_SHAPE;
    if (!device_is_sm103()) return FP8Q_ERR_UNSUPPORTED;
    if (a.M == 0) {  // no rows: the sums are zero, and nothing is added to what accumulates
        if (a.flags & FP8Q_ACCUMULATE) return FP8Q_OK;
        if (a.dweight && cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.N, stream) != cudaSuccess) return FP8Q_ERR_CUDA;
        if (a.dbias && cudaMemsetAsync(a.dbias, 0, sizeof(float) * a.N, stream) != cudaSuccess) return FP8Q_ERR_CUDA;
        return FP8Q_OK;
    }
    switch (a.dtype) {
        case FP8Q_BF16: return launch_bwd<__nv_bfloat16>(a, drop, stream);
        case FP8Q_FP16: return launch_bwd<__half>(a, drop, stream);
        default: return launch_bwd<float>(a, drop, stream);
    }
}
