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
// products of the columns are formed once.  The next rows' pieces are in flight
// in a ring of kRing rows in shared memory (norm_fwd.cuh); the generator is what
// bounds this kernel beside the memory, so no register holds a load in flight.
// SHIFT: rows off the 16-byte grid (norm_ops.cuh).
constexpr int kRing = 4;

template <typename T, bool RES, bool SHIFT>
__global__ void __launch_bounds__(256, 4) dropout_rows_kernel(const DropParams<T> p, int team, int chunks) {
    constexpr int V = 16 / sizeof(T), H = V / 2, kSlots = warp_slots(SHIFT, true), kStage = (RES ? 2 : 1) * kSlots;
    extern __shared__ uint4 s_ring[];  // [warp][stage][x, residual][slot]
    const int lane = threadIdx.x & 31;
    const int64_t N = p.N, pieces = SHIFT ? (N + V - 1) / V : N / V;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * blockDim.x >> 5;
    const int place = lane & (team - 1);
    const int first = static_cast<int>(warp % chunks) * 32;  // the warp's first piece
    const int rows_warp = 32 / team;
    const int64_t step = warps / chunks * rows_warp;  // rows that all warps of a chunk take at a time
    const int64_t left = N - static_cast<int64_t>(first + place) * V;  // columns from this thread's first
    const int valid_k = left <= 0 ? 0 : left < V ? static_cast<int>(left) : V;
    uint4* const ring = s_ring + (threadIdx.x >> 5) * (kRing * kStage) + lane + (SHIFT ? lane / team : 0);
    pdl_wait();
    if (warp / chunks >= warps / chunks) return;  // the warps that make no full set of chunks

    Philox g;
    uint64_t quad_m0 = 0;
    if (p.drop.on) {
        g = Philox(p.drop.rng);
        quad_m0 = kPhiloxM0 * (static_cast<uint32_t>(first + place) * (V / 4));
    }
    const int64_t bytes = (N - static_cast<int64_t>(first) * V) * static_cast<int64_t>(sizeof(T));  // of the row from `first` on
    auto fill_tensor = [&](uint4* to, const T* x, int64_t ld, int64_t row) {
        const T* start = x + row * ld + static_cast<int64_t>(first) * V;
        if constexpr (SHIFT)
            copy_granules(to, x, start, place, static_cast<int>(bytes < 1024 ? bytes : 1024), place == team - 1);
        else if (valid_k > 0)
            cp_async16(smem_u32(to), start + place * V);
    };
    auto fill = [&](int stage, int64_t row) {
        if (row < p.M) {
            fill_tensor(ring + stage * kStage, p.x, p.ldx, row);
            if constexpr (RES) fill_tensor(ring + stage * kStage + kSlots, p.res, p.ld_res, row);
        }
        cp_async_commit();
    };
    const int64_t base0 = warp / chunks * rows_warp;
    const int sub = lane / team;
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fill(k, base0 + sub + k * step);
    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
    int stage = 0;
    for (int64_t base = base0; base < p.M; base += step) {
        const int64_t row = base + sub;
        fill(stage == 0 ? kRing - 1 : stage - 1, row + (kRing - 1) * step);
        cp_async_wait<kRing - 1>();
        if constexpr (SHIFT) __syncwarp();
        const uint4* at = ring + stage * kStage;
        const int valid = row < p.M ? valid_k : 0;
        const T* x_row = p.x + row * p.ldx + static_cast<int64_t>(first) * V;
        Piece<T, V> x;
        x.raw = read_piece<SHIFT>(at, SHIFT ? granule_offset(x_row) : 0);
        f32x2 v[H];
        unpack2(x, v);
        if (p.drop.on) {
            uint32_t w[V];
            words_at<V>(g, quad_m0, g.row(static_cast<uint32_t>(row)), w);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = dropped2(mul2(v[i], inv2), w[2 * i], w[2 * i + 1], p.drop);
        }
        if constexpr (RES) {
            Piece<T, V> r;
            r.raw = read_piece<SHIFT>(at + kSlots, SHIFT ? granule_offset(p.res + row * p.ld_res + static_cast<int64_t>(first) * V) : 0);
            f32x2 f[H];
            unpack2(r, f);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = add2(f[i], v[i]);
        }
        pack2(x, v);
        T* y_row = p.y + row * p.ldy + static_cast<int64_t>(first) * V;
        if constexpr (SHIFT) {
            store_shifted<T>(x.raw, y_row, place, valid, team);
            __syncwarp();  // the granules that a neighbour read may be overwritten now
        } else if (valid > 0) {
            x.store(y_row + place * V);
        }
        stage = stage == kRing - 1 ? 0 : stage + 1;
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
}

template <typename T, bool RES, bool SHIFT>
cudaError_t launch_rows(const DropParams<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    static std::atomic<int> per_sm;  // CTAs that run at a time
    const auto kern = dropout_rows_kernel<T, RES, SHIFT>;
    const size_t smem = size_t(8) * kRing * (RES ? 2 : 1) * warp_slots(SHIFT, true) * 16;
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 256, smem);
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
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(256), smem, stream, p, team, static_cast<int>(chunks));
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
