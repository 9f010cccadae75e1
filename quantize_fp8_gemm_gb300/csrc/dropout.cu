// dropout.cu -- dropout_fwd and dropout_bwd: dropout from the counter-based
// generator of norm_ops.cuh, whose mask is formed where it is used and never
// stored, with the residual added in the same pass.
//
//     y  = T(float32(residual + (keep ? float32(x * inv) : 0)))
//     dx = keep ? T(float32(dy * inv)) : 0
#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>

namespace fp8q {

namespace {

template <typename T>
struct DropParams {
    int64_t M, N;
    const T* x;
    int64_t ldx;
    const T* res;
    int64_t ld_res;
    T* y;
    int64_t ldy;
    Dropout drop;
};

// Any layout: a thread takes quads of columns, one generator block each.
template <typename T>
__global__ void __launch_bounds__(256) dropout_quad_kernel(const DropParams<T> p) {
    pdl_wait();
    const int64_t quads = (p.N + 3) / 4, total = quads * p.M;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / quads, q = i - row * quads;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (p.drop.on) w = Philox(p.drop.rng).block(static_cast<uint32_t>(q), static_cast<uint32_t>(row));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t j = q * 4 + k;
            if (j >= p.N) continue;
            float v = to_f32(p.x[row * p.ldx + j]);
            if (p.drop.on) v = dropped(v, word_of(w, k), p.drop);
            if (p.res) v = __fadd_rn(to_f32(p.res[row * p.ld_res + j]), v);
            p.y[row * p.ldy + j] = from_f32<T>(v);
        }
    }
    pdl_launch_dependents();
}

// Division of n < 2^31 by a fixed d >= 1 as a product: n / d = (n * m) >> (31 + s)
// with s = ceil(log2 d), m = ceil(2^(31 + s) / d) (below 2^32); the excess
// n * (m d - 2^(31 + s)) / (d 2^(31 + s)) is below n / 2^31 / d < 1 / d, so
// the quotient is exact.
struct FastDiv {
    uint32_t m;
    int s;
    __host__ explicit FastDiv(uint32_t d) : s(31) {
        while ((1u << (s - 31)) < d) ++s;
        m = static_cast<uint32_t>(((uint64_t(1) << s) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> s);
    }
};

// Rows on the 16-byte grid: a thread takes U 16-byte pieces, loads first.
template <typename T, int U, bool RES>
__global__ void __launch_bounds__(256) dropout_piece_kernel(const DropParams<T> p, uint32_t total, uint32_t per_row,
                                                            const FastDiv div) {
    constexpr int V = 16 / sizeof(T);
    pdl_wait();
    const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
    Piece<T, V> x[U], r[U];
    uint32_t row[U], k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = first + u * 256u;
        row[u] = div.div(i);
        k[u] = i - row[u] * per_row;
        if (i < total) x[u].load(p.x + static_cast<int64_t>(row[u]) * p.ldx + static_cast<int64_t>(k[u]) * V);
    }
    if constexpr (RES) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (first + u * 256u < total)
                r[u].load(p.res + static_cast<int64_t>(row[u]) * p.ld_res + static_cast<int64_t>(k[u]) * V);
    }
    Philox g;
    if (p.drop.on) g = Philox(p.drop.rng);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (first + u * 256u >= total) continue;
        float v[V];
        x[u].unpack(v);
        if (p.drop.on) {
            uint32_t w[V];
            words_at<V>(g, k[u] * V, row[u], w);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = dropped(v[i], w[i], p.drop);
        }
        if constexpr (RES) {
            float f[V];
            r[u].unpack(f);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __fadd_rn(f[i], v[i]);
        }
        x[u].pack(v);
        x[u].store(p.y + static_cast<int64_t>(row[u]) * p.ldy + static_cast<int64_t>(k[u]) * V);
    }
    pdl_launch_dependents();
}

template <typename T>
int launch_drop(const void* x, int64_t ldx, const void* res, int64_t ld_res, void* y, int64_t ldy, int64_t M, int64_t N,
                const Dropout& drop, cudaStream_t stream) {
    const DropParams<T> p = {M, N, static_cast<const T*>(x), ldx, static_cast<const T*>(res), ld_res,
                             static_cast<T*>(y), ldy, drop};
    constexpr int V = 16 / sizeof(T), U = 2;
    if (N % V == 0 && rows16(x, ldx, sizeof(T)) && rows16(res, ld_res, sizeof(T)) && rows16(y, ldy, sizeof(T)) &&
        N / V < (int64_t(1) << 31) / M) {
        const uint32_t per_row = static_cast<uint32_t>(N / V), total = per_row * static_cast<uint32_t>(M);
        const dim3 grid((total + 256 * U - 1) / (256 * U));
        const FastDiv div(per_row);
        if ((res ? launch_pdl(dropout_piece_kernel<T, U, true>, grid, dim3(256), 0, stream, p, total, per_row, div)
                 : launch_pdl(dropout_piece_kernel<T, U, false>, grid, dim3(256), 0, stream, p, total, per_row, div)) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return FP8Q_ERR_CUDA;
        }
        return FP8Q_OK;
    }
    const int64_t want = ((N + 3) / 4 * M + 255) / 256;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, int64_t(sm_count()) * 64));
    if (launch_pdl(dropout_quad_kernel<T>, dim3(grid), dim3(256), 0, stream, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return FP8Q_OK;
}

int run_drop(const void* x, int64_t ldx, const void* res, int64_t ld_res, void* y, int64_t ldy, int64_t M, int64_t N,
             int dtype, double prob, const uint64_t* rng, cudaStream_t stream) {
    if (!is_dtype(dtype)) return FP8Q_ERR_UNSUPPORTED;
    if (M < 0 || N < 1 || M > FP8Q_NORM_MAX || N > FP8Q_NORM_MAX) return FP8Q_ERR_SHAPE;
    Dropout drop;
    if (!make_dropout(prob, rng, &drop)) return FP8Q_ERR_SHAPE;
    if (M > 0 && (!x || !y || (drop.on && !rng))) return FP8Q_ERR_NULL;
    if (ldx < N || ldy < N || (res && ld_res < N)) return FP8Q_ERR_SHAPE;
    const size_t es = dtype_size(dtype);
    if (!aligned_to(x, es) || !aligned_to(res, es) || !aligned_to(y, es) || !aligned_to(rng, 8)) return FP8Q_ERR_ALIGN;
    if (!device_is_sm103()) return FP8Q_ERR_UNSUPPORTED;
    if (M == 0) return FP8Q_OK;
    switch (dtype) {
        case FP8Q_BF16: return launch_drop<__nv_bfloat16>(x, ldx, res, ld_res, y, ldy, M, N, drop, stream);
        case FP8Q_FP16: return launch_drop<__half>(x, ldx, res, ld_res, y, ldy, M, N, drop, stream);
        default: return launch_drop<float>(x, ldx, res, ld_res, y, ldy, M, N, drop, stream);
    }
}

}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" int dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ld_residual, void* y, int64_t ldy,
                           int64_t M, int64_t N, int dtype, double p, const uint64_t* rng, cudaStream_t stream) {
    return run_drop(x, ldx, residual, ld_residual, y, ldy, M, N, dtype, p, rng, stream);
}

extern "C" int dropout_bwd(const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx, int64_t M, int64_t N, int dtype,
                           double p, const uint64_t* rng, cudaStream_t stream) {
    return run_drop(dy, ld_dy, nullptr, 0, dx, ld_dx, M, N, dtype, p, rng, stream);
}
