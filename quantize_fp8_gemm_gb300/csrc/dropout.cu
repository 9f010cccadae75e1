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
// 1600 159 us (0.78 of the measured copy rate), with residual 205 us (0.90);
// 65536 x 768 with residual 52 us (0.85); float32 65536 x 1600 129 us (0.96).  Off
// the 16-byte grid the instructions of single elements come on top (112 for 128
// elements, 138 with residual; the integer pipe at 57 and 62 % of its cycles):
// 65536 x 1601 with residual 167 us (0.55), float32 65536 x 1001 with residual 122 us
// (0.95), without 103 us (0.75).
#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>
#include <type_traits>

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
// 159 at 4 (the generator's chains hide each other); float32 65536 x 1600 156, 131, 135.
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

// Rows off the 16-byte grid, or too many pieces for 31 bits.  A warp takes 128 columns
// (or, where rows have at most 64, 32 / team rows), the same of each row that it
// comes to, U of them at a time, loads first.  A lane forms the block of one column
// quad, but loads and stores single elements, 32 adjacent ones a warp: a tensor may
// begin anywhere, and each access is of whole sectors but at its ends.  The mask goes
// from the quads to the elements by four votes: bit q of vote i is element 4q + i.
// (Pieces of eight elements, cut from aligned granules in shared memory and joined
// into such, took 230 us at 65536 x 1601 with residual, 155 us at float32 65536 x
// 1001, 7.2 us at fp16 4097 x 333; this takes 167, 103 and 3.6.)
//
// Rows at a time, where rows are wide: with residual 65536 x 1601 takes 203 us at 2 and
// three CTAs a multiprocessor, 166 at 3, 162 to 167 at 4, 178 at 6.  Narrow ones hold
// four addresses a tensor: what fits the registers (131072 x 63: 14 us at 2, 19 at 4).
template <bool RES, bool NARROW>
constexpr int kRows = NARROW ? (RES ? 1 : 2) : 4;

template <typename T, bool RES, bool NARROW>
__global__ void __launch_bounds__(256, 2) dropout_elems_kernel(const DropParams<T> p, int team, uint32_t spans) {
    constexpr uint32_t U = kRows<RES, NARROW>;
    const int lane = threadIdx.x & 31;
    const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
    const uint32_t set = warp / spans, sets = warps / spans, span = warp - set * spans;
    pdl_wait();
    if (set >= sets) return;  // the warps that make no full set
    const uint32_t per = NARROW ? 32 / team : 1;  // rows a warp at a time
    const uint32_t M = static_cast<uint32_t>(p.M), step = sets * per;
    const int64_t first = static_cast<int64_t>(span) * 128, columns = p.N - first;
    uint32_t row = set * per;
    bool in[4];
    uint32_t sub[4];
    int64_t xo[4], ro[4], yo[4];  // of an element from its warp's first; past the row's end the last one's
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int q = 8 * s + (lane >> 2);  // the quad of element s
        sub[s] = NARROW ? q / team : 0;
        int c = NARROW ? 4 * (q & (team - 1)) + (lane & 3) : 32 * s + lane;
        in[s] = c < columns;
        if (!in[s]) c = static_cast<int>(columns) - 1;
        xo[s] = sub[s] * p.ldx + c;
        ro[s] = sub[s] * p.ld_res + c;
        yo[s] = sub[s] * p.ldy + c;
    }
    const T* x = p.x + row * p.ldx + first;
    const T* res = RES ? p.res + row * p.ld_res + first : nullptr;
    T* y = p.y + row * p.ldy + first;
    const int64_t x_step = step * p.ldx, r_step = step * p.ld_res, y_step = step * p.ldy;
    const uint32_t own = NARROW ? lane / team : 0;  // the row of this lane's quad among the warp's
    Philox g;
    uint64_t quad_m0 = 0;
    if (p.drop.on) {
        g = Philox(p.drop.rng);
        quad_m0 = kPhiloxM0 * (span * 32 + (NARROW ? lane & (team - 1) : lane));
    }
    // n: rows (of this warp, `step` apart) that the batch has, 1 .. U
    auto batch = [&](auto full, uint32_t n) {
        constexpr bool FULL = decltype(full)::value;
        T v[U][4], f[U][4];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t at = FULL ? u : min(u, n - 1);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (NARROW && sub[s] >= M - row - at * step)
                    v[u][s] = f[u][s] = from_f32<T>(0.0f);
                else {
                    v[u][s] = x[at * x_step + xo[s]];
                    if constexpr (RES) f[u][s] = res[at * r_step + ro[s]];
                }
            }
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (!FULL && u == n) break;
            uint32_t keep = ~0u;
            if (p.drop.on) {
                const uint4 w = g.block(quad_m0, g.row(row + u * step + own));
                const uint32_t k0 = __ballot_sync(~0u, w.x > p.drop.last), k1 = __ballot_sync(~0u, w.y > p.drop.last),
                               k2 = __ballot_sync(~0u, w.z > p.drop.last), k3 = __ballot_sync(~0u, w.w > p.drop.last);
                const uint32_t even = lane & 2 ? k2 : k0, odd = lane & 2 ? k3 : k1;
                keep = (lane & 1 ? odd : even) >> (lane >> 2);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float o = to_f32(v[u][s]) * p.drop.inv;
                o = keep & (1u << (8 * s)) ? o : 0.0f;
                if constexpr (RES) o = to_f32(f[u][s]) + o;
                if (in[s] && (!NARROW || sub[s] < M - row - u * step)) y[u * y_step + yo[s]] = from_f32<T>(o);
            }
        }
        row += U * step;
        x += U * x_step;
        if constexpr (RES) res += U * r_step;
        y += U * y_step;
    };
    uint32_t n = row < M ? (M - row + step - 1) / step : 0;
    for (; n >= U; n -= U) batch(std::true_type(), U);
    if (n != 0) batch(std::false_type(), n);
    pdl_launch_dependents();
}

template <typename T, bool RES, bool NARROW>
cudaError_t launch_elems(const DropParams<T>& p, int team, cudaStream_t stream) {
    static DeviceTable<17> table;  // CTAs that run at a time
    const auto kern = dropout_elems_kernel<T, RES, NARROW>;
    int n = 0;
    const cudaError_t e = resident_ctas(table, kern, 256, 0, 0, &n);
    if (e != cudaSuccess) return e;
    const int64_t spans = (p.N + 127) / 128, rows = (p.M + 32 / team - 1) / (32 / team);
    const int64_t want = (rows * spans + 7) / 8, least = (spans + 7) / 8;  // least: one full set of a row's warps
    const int64_t grid = std::max(least, std::min<int64_t>(want, int64_t(n) * sm_count()));
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, p, team,
                      static_cast<uint32_t>(spans));
}

template <typename T, bool RES>
cudaError_t launch_rows(const DropParams<T>& p, cudaStream_t stream) {
    const int team = team_of((p.N + 3) / 4);
    return team < 32 ? launch_elems<T, RES, true>(p, team, stream) : launch_elems<T, RES, false>(p, team, stream);
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
