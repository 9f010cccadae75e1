// dropout.cu -- dropout_fwd and dropout_bwd: dropout from the counter-based
// generator of norm_ops.cuh, whose mask is formed where it is used and never
// stored, with the residual added in the same pass.
//
//     y  = T(float32(residual + (keep ? float32(x * inv) : 0)))
//     dx = keep ? T(float32(dy * inv)) : 0
//
// What bounds it: memory beside the generator's multiplications.  The 17 products
// of a block (norm_ops.cuh) keep the multiply pipe at 60 to 70 % of its cycles, at
// which it is full beside the other instructions.  Measured on GB300: bf16 131072 x
// 1600 160 us (0.77 of the measured copy rate), with residual 205 us (0.90);
// 65536 x 768 with residual 52 us (0.85); float32 65536 x 1600 129 us (0.96).  Off
// the 16-byte grid 65536 x 1601 with residual 229 us (0.40).
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

// Division of n < 2^31 by a fixed d >= 1 as a product: n / d = (n * m) >> s with
// s = 31 + ceil(log2 d), m = ceil(2^s / d) (below 2^32); the excess of n m / 2^s
// over n / d is n (m d - 2^s) / (d 2^s) < n / 2^31 / d < 1 / d, so the quotient
// is exact.
struct FastDiv {
    uint32_t m;
    int s;
    explicit FastDiv(uint32_t d) : s(31) {
        while ((1u << (s - 31)) < d) ++s;
        m = static_cast<uint32_t>(((uint64_t(1) << s) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> s);
    }
};

// Pieces a thread: 131072 x 1600 bf16 without residual takes 193 us at 1, 169 at 2,
// 160 at 4 (the generator's chains hide each other); float32 65536 x 1600 156, 131, 135.
template <typename T>
constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;

// Rows on the 16-byte grid: a thread takes U 16-byte pieces, loads first.
// FLAT: the tensors are packed, so that a piece's place is its number.
template <typename T, bool RES, bool FLAT>
__global__ void __launch_bounds__(256) dropout_pieces_kernel(const DropParams<T> p, uint32_t total, uint32_t per_row,
                                                             const FastDiv div) {
    constexpr int V = 16 / sizeof(T), H = V / 2, U = kUnroll<T>;
    pdl_wait();
    const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
    Piece<T, V> x[U], r[U];
    uint32_t row[U], k[U];
    auto at = [&](int u, int64_t ld) {
        return FLAT ? static_cast<int64_t>(first + u * 256u) * V
                    : static_cast<int64_t>(row[u]) * ld + static_cast<int64_t>(k[u]) * V;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = first + u * 256u;
        row[u] = div.div(i);
        k[u] = i - row[u] * per_row;
        x[u].zero();
        if (i < total) x[u].load(p.x + at(u, p.ldx));
    }
    if constexpr (RES) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u].zero();
            if (first + u * 256u < total) r[u].load(p.res + at(u, p.ld_res));
        }
    }
    Philox g;
    if (p.drop.on) g = Philox(p.drop.rng);
    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        f32x2 v[H];
        unpack2(x[u], v);
        if (p.drop.on) {
            uint32_t w[V];
            words_at<V>(g, kPhiloxM0 * (k[u] * (V / 4)), g.row(row[u]), w);
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
        if (first + u * 256u < total) x[u].store(p.y + at(u, p.ldy));
    }
    pdl_launch_dependents();
}

template <typename T>
cudaError_t launch_pieces(const DropParams<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const uint32_t per_row = static_cast<uint32_t>(p.N / V), total = per_row * static_cast<uint32_t>(p.M);
    const dim3 grid((total + 256 * kUnroll<T> - 1) / (256 * kUnroll<T>));
    const FastDiv div(per_row);
    const bool flat = p.ldx == p.N && p.ldy == p.N && (!p.res || p.ld_res == p.N);
    const auto kern = p.res ? (flat ? dropout_pieces_kernel<T, true, true> : dropout_pieces_kernel<T, true, false>)
                            : (flat ? dropout_pieces_kernel<T, false, true> : dropout_pieces_kernel<T, false, false>);
    return launch_pdl(kern, grid, dim3(256), 0, stream, p, total, per_row, div);
}

// Rows off the 16-byte grid (norm_ops.cuh), or too many pieces for 31 bits.  A warp
// takes `deep` runs of 32 adjacent pieces of a row (or, where a row has
// fewer than 32, 32 / team rows), the same columns of every row that it comes to.
// The next runs are in flight in a ring of kRing in shared memory (norm_fwd.cuh);
// the generator is what bounds this kernel beside the memory, so no register holds
// a load in flight.
constexpr int kRing = 4;

template <typename T, bool RES>
__global__ void __launch_bounds__(256, 4) dropout_rows_kernel(const DropParams<T> p, int team, int chunks, int deep) {
    constexpr int V = 16 / sizeof(T), H = V / 2, kSlots = warp_slots(true, true), kStage = (RES ? 2 : 1) * kSlots;
    extern __shared__ uint4 s_ring[];  // [warp][stage][x, residual][slot]
    const int lane = threadIdx.x & 31, place = lane & (team - 1);
    const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
    const uint32_t parts = static_cast<uint32_t>((chunks + deep - 1) / deep);  // warps that a row takes
    const uint32_t set = warp / parts, sets = warps / parts;
    const int first = static_cast<int>(warp - set * parts) * deep, runs = min(deep, chunks - first);  // this one's runs of it
    const uint32_t step = sets * (32 / team);  // rows that all warps take at a time
    uint4* const ring = s_ring + (threadIdx.x >> 5) * (kRing * kStage) + lane + lane / team;
    pdl_wait();
    if (set >= sets) return;  // the warps that make no full set

    const int64_t left = p.N - (static_cast<int64_t>(first) * 32 + place) * V;  // columns from this thread's first
    Philox g;
    uint64_t first_m0 = 0;
    if (p.drop.on) {
        g = Philox(p.drop.rng);
        first_m0 = kPhiloxM0 * ((static_cast<uint32_t>(first) * 32 + place) * (V / 4));
    }
    const uint32_t M = static_cast<uint32_t>(p.M);
    uint32_t base = set * (32 / team), row = base + lane / team;
    const int64_t column = static_cast<int64_t>(first) * 32 * V;
    const T *x_at = p.x + static_cast<int64_t>(row) * p.ldx + column, *r_at = p.res + static_cast<int64_t>(row) * p.ld_res + column;
    T* y_at = p.y + static_cast<int64_t>(row) * p.ldy + column;
    const int64_t x_step = step * p.ldx, r_step = step * p.ld_res, y_step = step * p.ldy;
    const uint32_t ring_at = smem_u32(ring);

    // what is put in flight next: run `run_in` of row `row_in`
    const T *x_in = x_at, *r_in = r_at;
    uint32_t row_in = row;
    int run_in = 0;
    auto fill_tensor = [&](uint32_t to, const T* start) {
        const int64_t rest = left - static_cast<int64_t>(run_in) * 32 * V;
        const uint32_t mis = granule_offset(start);
        const int64_t bytes = (rest + place * V) * static_cast<int64_t>(sizeof(T)) + mis;  // from the run's first granule on
        copy_granules<false>(to, reinterpret_cast<const uint8_t*>(start + run_in * 32 * V) - mis, place,
                             static_cast<int>(bytes < 1024 ? bytes : 1024), place == team - 1);
    };
    auto fill = [&](int stage) {
        if (row_in < M) {
            fill_tensor(ring_at + stage * kStage * 16, x_in);
            if constexpr (RES) fill_tensor(ring_at + (stage * kStage + kSlots) * 16, r_in);
        }
        cp_async_commit();
        if (++run_in == runs) {
            run_in = 0;
            row_in += step;
            x_in += x_step;
            if constexpr (RES) r_in += r_step;
        }
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fill(k);
    const f32x2 inv2 = pair_of(p.drop.inv, p.drop.inv);
    uint4 carry = make_uint4(0, 0, 0, 0);
    int stage = 0, run = 0;
    uint64_t row_m0 = p.drop.on ? g.row(row) : 0, quad_m0 = first_m0;
    while (base < M) {
        fill(stage == 0 ? kRing - 1 : stage - 1);
        cp_async_wait<kRing - 1>();
        __syncwarp();
        const uint4* at = ring + stage * kStage;
        Piece<T, V> x;
        x.raw = read_piece<T, true>(at, granule_offset(x_at));
        f32x2 v[H];
        unpack2(x, v);
        if (p.drop.on) {
            uint32_t w[V];
            words_at<V>(g, quad_m0, row_m0, w);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = dropped2(mul2(v[i], inv2), w[2 * i], w[2 * i + 1], p.drop);
        }
        if constexpr (RES) {
            Piece<T, V> r;
            r.raw = read_piece<T, true>(at + kSlots, granule_offset(r_at));
            f32x2 f[H];
            unpack2(r, f);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = add2(f[i], v[i]);
        }
        pack2(x, v);
        const int64_t rest = row < M ? left - static_cast<int64_t>(run) * 32 * V : 0;
        const int valid = rest <= 0 ? 0 : rest < V ? static_cast<int>(rest) : V;
        if (run > 0 && run < runs - 1)
            store_shifted<T, false, false>(x.raw, carry, y_at, run * 32 + place, valid, false, false);
        else
            store_shifted<T, true, true>(x.raw, carry, y_at, run * 32 + place, valid, run == 0 && place == 0,
                                         rest <= V || (run == runs - 1 && place == 31));
        __syncwarp();  // the granules that a neighbour read may be overwritten now
        stage = stage == kRing - 1 ? 0 : stage + 1;
        quad_m0 += kPhiloxM0 * (32 * (V / 4));
        if (++run == runs) {
            run = 0;
            base += step;
            row += step;
            x_at += x_step;
            if constexpr (RES) r_at += r_step;
            y_at += y_step;
            quad_m0 = first_m0;
            if (p.drop.on) row_m0 = g.row(row);
        }
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
}

template <typename T, bool RES>
cudaError_t launch_rows(const DropParams<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    static std::atomic<int> per_sm;  // CTAs that run at a time
    const auto kern = dropout_rows_kernel<T, RES>;
    const size_t smem = size_t(8) * kRing * (RES ? 2 : 1) * warp_slots(true, true) * 16;
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 256, smem);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
        per_sm.store(n, std::memory_order_relaxed);
    }
    const int64_t pieces = (p.N + V - 1) / V, chunks = (pieces + 31) / 32;
    const int team = team_of(pieces);
    const int64_t rows = (p.M + 32 / team - 1) / (32 / team);
    // a warp's part of a row has ends that go element by element: up to 8 runs a part,
    // where that leaves two rows a warp
    int64_t deep = 1;
    while (deep < 8 && deep < chunks && rows * ((chunks + 2 * deep - 1) / (2 * deep)) >= int64_t(n) * sm_count() * 16) deep *= 2;
    const int64_t parts = (chunks + deep - 1) / deep;
    const int64_t want = (rows * parts + 7) / 8, least = (parts + 7) / 8;  // least: one full set of a row's warps
    const int64_t grid = std::max(least, std::min<int64_t>(want, int64_t(n) * sm_count()));
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(256), smem, stream, p, team, static_cast<int>(chunks),
                      static_cast<int>(deep));
}

template <typename T>
int launch_drop(const void* x, int64_t ldx, const void* res, int64_t ld_res, void* y, int64_t ldy, int64_t M, int64_t N,
                const Dropout& drop, cudaStream_t stream) {
    const DropParams<T> p = {M, N, static_cast<const T*>(x), ldx, static_cast<const T*>(res), ld_res,
                             static_cast<T*>(y), ldy, drop};
    constexpr int V = 16 / sizeof(T);
    cudaError_t e;
    if (N % V == 0 && rows16(x, ldx, sizeof(T)) && rows16(res, ld_res, sizeof(T)) && rows16(y, ldy, sizeof(T)) &&
        N / V < (int64_t(1) << 31) / M)
        e = launch_pieces<T>(p, stream);
    else
        e = res ? launch_rows<T, true>(p, stream) : launch_rows<T, false>(p, stream);
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
