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
    // of the row from `first` on: as many bytes as the warp's granules can hold, or fewer
    const int64_t rest = (N - static_cast<int64_t>(first) * V) * static_cast<int64_t>(sizeof(T));
    const int bytes = static_cast<int>(rest < 1024 ? rest : 1024);
    const uint32_t M = static_cast<uint32_t>(p.M), steps = static_cast<uint32_t>(step);
    uint32_t base = static_cast<uint32_t>(warp / chunks * rows_warp), row = base + lane / team, next = row;
    const int64_t at0 = static_cast<int64_t>(row), column = static_cast<int64_t>(first) * V;
    const T *x_in = p.x + at0 * p.ldx + column, *r_in = p.res + at0 * p.ld_res + column, *x_at = x_in, *r_at = r_in;
    T* y_at = p.y + at0 * p.ldy + column;
    const int64_t x_step = step * p.ldx, r_step = step * p.ld_res, y_step = step * p.ldy;
    const uint32_t ring_at = smem_u32(ring);
    auto fill_tensor = [&](uint32_t to, const T* base_of, const T* start) {
        if constexpr (SHIFT)
            copy_granules(to, base_of, start, place, bytes, place == team - 1);
        else if (valid_k > 0)
            cp_async16(to, start + place * V);
    };
    // the next row that is to be in flight, into a stage; nothing past the last row
    auto fill = [&](int stage) {
        if (next < M) {
            fill_tensor(ring_at + stage * kStage * 16, p.x, x_in);
            if constexpr (RES) fill_tensor(ring_at + (stage * kStage + kSlots) * 16, p.res, r_in);
        }
        cp_async_commit();
        next += steps;
        x_in += x_step;
        if constexpr (RES) r_in += r_step;
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fill(k);
    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
    uint4 carry = make_uint4(0, 0, 0, 0);
    int stage = 0;
    for (; base < M; base += steps) {
        fill(stage == 0 ? kRing - 1 : stage - 1);
        cp_async_wait<kRing - 1>();
        if constexpr (SHIFT) __syncwarp();
        const uint4* at = ring + stage * kStage;
        Piece<T, V> x;
        x.raw = read_piece<SHIFT>(at, SHIFT ? granule_offset(x_at) : 0);
        f32x2 v[H];
        unpack2(x, v);
        if (p.drop.on) {
            uint32_t w[V];
            words_at<V>(g, quad_m0, g.row(row), w);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = dropped2(mul2(v[i], inv2), w[2 * i], w[2 * i + 1], p.drop);
        }
        if constexpr (RES) {
            Piece<T, V> r;
            r.raw = read_piece<SHIFT>(at + kSlots, SHIFT ? granule_offset(r_at) : 0);
            f32x2 f[H];
            unpack2(r, f);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = add2(f[i], v[i]);
        }
        pack2(x, v);
        const int valid = row < M ? valid_k : 0;
        if constexpr (SHIFT) {
            store_shifted<T>(x.raw, carry, y_at, place, valid, place == 0, place == 31 || first + place == pieces - 1);
            __syncwarp();  // the granules that a neighbour read may be overwritten now
        } else if (valid > 0) {
            x.store(y_at + place * V);
        }
        stage = stage == kRing - 1 ? 0 : stage + 1;
        row += steps;
        x_at += x_step;
        if constexpr (RES) r_at += r_step;
        y_at += y_step;
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
