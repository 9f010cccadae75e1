// dropout.cu -- dropout_fwd and dropout_bwd: dropout from the counter-based
// generator of norm_ops.cuh, whose mask is formed where it is used and never
// stored, with the residual added in the same pass.
//
//     y  = T(float32(residual + (keep ? float32(x * inv) : 0)))
//     dx = keep ? T(float32(dy * inv)) : 0
#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>
#include <atomic>

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

// A warp takes 32 adjacent pieces of a row (or, where a row has fewer, 32 / team
// rows), the same columns of every row that it comes to: the generator's
// products of the columns are formed once.  U rows are in flight a warp.
// SHIFT: rows off the 16-byte grid (norm_ops.cuh); a lane loads the two granules
// that hold its piece (the second from L1, where its neighbour brought it).
template <typename T, bool RES, bool SHIFT>
__global__ void __launch_bounds__(256, 4) dropout_rows_kernel(const DropParams<T> p, int team, int chunks) {
    constexpr int V = 16 / sizeof(T), H = V / 2, U = 2;
    const int lane = threadIdx.x & 31;
    const int64_t N = p.N, pieces = SHIFT ? (N + V - 1) / V : N / V;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * blockDim.x >> 5;
    const int k = static_cast<int>(warp % chunks) * 32 + (lane & (team - 1));
    const int rows_warp = 32 / team;
    const int64_t step = warps / chunks * rows_warp;  // rows that all warps of a chunk take at a time
    const int64_t first = warp / chunks * rows_warp + lane / team;
    const int64_t left = N - static_cast<int64_t>(k) * V;  // columns from this thread's first
    const int valid_k = k < pieces ? (left < V ? static_cast<int>(left) : V) : 0;
    pdl_wait();
    if (warp / chunks >= warps / chunks) return;  // the warps that make no full set of chunks

    Philox g;
    uint64_t quad_m0 = 0;
    if (p.drop.on) {
        g = Philox(p.drop.rng);
        quad_m0 = kPhiloxM0 * (static_cast<uint32_t>(k) * (V / 4));
    }
    auto load = [&](const T* start, bool in) -> uint4 {
        if constexpr (SHIFT) {
            const uint32_t mis = granule_offset(start);
            const uint4* at = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(start) - mis) + k;
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (in) a = __ldg(at);
            if (in && (k + int64_t(1)) * 16 - mis < N * static_cast<int64_t>(sizeof(T))) b = __ldg(at + 1);
            return cut16(a, b, mis);
        } else {
            return in ? ld_stream_v4(start + static_cast<int64_t>(k) * V) : make_uint4(0, 0, 0, 0);
        }
    };
    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
    for (int64_t base = first - lane / team; base < p.M; base += U * step) {
        Piece<T, V> x[U], r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + lane / team + u * step;
            const bool in = row < p.M && valid_k > 0;
            x[u].raw = load(p.x + (in ? row : 0) * p.ldx, in);
            if constexpr (RES) r[u].raw = load(p.res + (in ? row : 0) * p.ld_res, in);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + lane / team + u * step;
            const int valid = row < p.M ? valid_k : 0;
            if (!SHIFT && valid == 0) continue;
            f32x2 v[H];
            unpack2(x[u], v);
            if (p.drop.on) {
                uint32_t w[V];
                words_at<V>(g, quad_m0, g.row(static_cast<uint32_t>(row)), w);
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = dropped2(mul2(v[i], inv2), w[2 * i], w[2 * i + 1], p.drop);
            }
            if constexpr (RES) {
                f32x2 f[H];
                unpack2(r[u], f);
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = add2(f[i], v[i]);
            }
            pack2(x[u], v);
            if constexpr (SHIFT) store_shifted<T>(x[u].raw, p.y + row * p.ldy, k, valid, team);
            else x[u].store(p.y + row * p.ldy + static_cast<int64_t>(k) * V);
        }
    }
    pdl_launch_dependents();
}

template <typename T, bool RES, bool SHIFT>
cudaError_t launch_rows(const DropParams<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    static std::atomic<int> per_sm;  // CTAs that run at a time
    const auto kern = dropout_rows_kernel<T, RES, SHIFT>;
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 256, 0);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
        per_sm.store(n, std::memory_order_relaxed);
    }
    const int64_t pieces = (p.N + V - 1) / V;
    const int team = team_of(pieces);
    const int64_t chunks = (pieces + 31) / 32, rows_warp = 32 / team;
    const int64_t want = ((p.M + rows_warp - 1) / rows_warp * chunks + 7) / 8;
    const int64_t least = (chunks + 7) / 8;  // one full set of chunks
    const int64_t grid = std::max(least, std::min<int64_t>(want, int64_t(n) * sm_count()));
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, p, team, static_cast<int>(chunks));
}

template <typename T>
int launch_drop(const void* x, int64_t ldx, const void* res, int64_t ld_res, void* y, int64_t ldy, int64_t M, int64_t N,
                const Dropout& drop, cudaStream_t stream) {
    const DropParams<T> p = {M, N, static_cast<const T*>(x), ldx, static_cast<const T*>(res), ld_res,
                             static_cast<T*>(y), ldy, drop};
    constexpr int V = 16 / sizeof(T);
    cudaError_t e;
    if (N % V == 0 && rows16(x, ldx, sizeof(T)) && rows16(res, ld_res, sizeof(T)) && rows16(y, ldy, sizeof(T)))
        e = res ? launch_rows<T, true, false>(p, stream) : launch_rows<T, false, false>(p, stream);
    else
        e = res ? launch_rows<T, true, true>(p, stream) : launch_rows<T, false, true>(p, stream);
    if (e != cudaSuccess) {
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
