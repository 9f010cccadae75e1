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
#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>
#include <atomic>

namespace fp8q {

namespace {

template <typename T>
struct BwdParams {
    int64_t M, N;
    const T* dy;
    int64_t ld_dy;
    const T* r;
    int64_t ld_r;
    const float* mean;
    const float* rstd;
    Params<T> w;
    const T* dres;
    int64_t ld_dres;
    T* dx;
    int64_t ld_dx;
    T* dbranch;
    int64_t ld_db;
    Dropout drop;
    float* part;  // [parts][2][N]: dweight and dbias sums of a set of rows
    int parts;
};

// Any width: one CTA per row, two passes over it.
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
                w = Philox(p.drop.rng).block(static_cast<uint32_t>(q), static_cast<uint32_t>(row));
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
// columns; warp k of its 32 adds parts k, k + 32, ..., then the warps' sums are
// added in order.
__global__ void __launch_bounds__(1024) ln_bwd_reduce_kernel(const float* part, int parts, int64_t N, float* dweight,
                                                             float* dbias, bool accumulate) {
    __shared__ float s[32][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // column of [2][N]
    float sum = 0.0f;
    if (j < 2 * N) {
#pragma unroll 4
        for (int k = warp; k < parts; k += 32) sum += part[static_cast<int64_t>(k) * 2 * N + j];
    }
    s[warp][lane] = sum;
    __syncthreads();
    sum = s[lane][warp];  // column `warp` of the block
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
    if (lane == 0 && col < 2 * N) {
        float* out = col < N ? dweight : dbias;
        if (out) {
            out += col < N ? col : col - N;
            *out = accumulate ? *out + sum : sum;
        }
    }
    pdl_launch_dependents();
}

// One pass: every input is read once.  A thread keeps its C pieces' columns for
// all the rows that its CTA takes (row blockIdx.x, + the grid, ...), so the
// column sums stay in registers until the end.  16-byte pieces come through a
// ring of kStages rows in shared memory, filled by cp.async: a thread copies
// and reads its own pieces only, so it waits for its own copies and no barrier
// guards the ring.  Single elements are loaded where they are used.
enum RowsMode {
    NARROW,  // `team` lanes (a power of two) take a row, 32 / team rows a warp, 4 warps
    WIDE,    // a CTA of up to 512 threads takes a row
    BROAD    // the same with up to 1024 threads, whose 64 registers hold no weights
};

// Rows of the ring: what a CTA's shared memory holds of its widest row.  A
// stage is 48 C bytes a thread: 96 KB for 512 threads of C = 4, or 1024 of C = 2.
constexpr int ring_stages(int V, int C, RowsMode mode) {
    return V == 1 ? 0 : mode == BROAD ? (C == 4 ? 1 : 2) : mode == WIDE && C == 4 ? 2 : 3;
}

template <typename T, int V, int C, RowsMode MODE, bool DROP>
__global__ void __launch_bounds__(MODE == NARROW ? 128 : MODE == WIDE ? 512 : 1024)
ln_bwd_rows_kernel(const BwdParams<T> p, int team) {
    extern __shared__ uint4 s_ring[];  // [stage][dy, r, dresidual][c][thread]
    __shared__ float s_part[MODE == NARROW ? 2 * 32 * C * V : 1];
    __shared__ float2 s_sum[2][32];
    constexpr int S = ring_stages(V, C, MODE);
    constexpr bool kHeld = V > 1 && MODE != BROAD;  // weights in registers
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int t = MODE == NARROW ? lane & (team - 1) : threadIdx.x;
    const int span = MODE == NARROW ? team : blockDim.x;
    const int pieces = static_cast<int>(p.N / V);
    const float inv_n = 1.0f / static_cast<float>(p.N);
    pdl_wait();

    float w[kHeld ? C : 1][V], dw[C][V], db[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < V; ++i) dw[c][i] = db[c][i] = 0.0f;
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[c][i] = 0.0f;
            if (t + c * span < pieces) load_params<T, V>(p.w, static_cast<int64_t>(t + c * span) * V, w[c]);
        }
    }
    Philox g;
    if constexpr (DROP) g = Philox(p.drop.rng);

    const int rows_warp = MODE == NARROW ? 32 / team : 1;
    const int rows_cta = MODE == NARROW ? rows_warp * nw : 1;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_cta;
    const int64_t base0 = static_cast<int64_t>(blockIdx.x) * rows_cta;
    const int64_t sub = MODE == NARROW ? warp * rows_warp + lane / team : 0;

    // pieces past the row, and rows past the last, are zeros
    auto slot = [&](int stage, int tensor, int c) {
        return s_ring + ((stage * 3 + tensor) * C + c) * static_cast<int>(blockDim.x) + threadIdx.x;
    };
    auto fill = [&](int stage, int64_t row) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool in = row < p.M && t + c * span < pieces;
            const int64_t j = static_cast<int64_t>(t + c * span) * V;
            cp_async16_or_zero(smem_u32(slot(stage, 0, c)), in ? p.dy + row * p.ld_dy + j : p.dy, in);
            cp_async16_or_zero(smem_u32(slot(stage, 1, c)), in ? p.r + row * p.ld_r + j : p.r, in);
            if (p.dres) cp_async16_or_zero(smem_u32(slot(stage, 2, c)), in ? p.dres + row * p.ld_dres + j : p.dres, in);
        }
        cp_async_commit();
    };
    if constexpr (S > 0) {
#pragma unroll
        for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);
    }
    float mean = base0 + sub < p.M ? p.mean[base0 + sub] : 0.0f;
    float rstd = base0 + sub < p.M ? p.rstd[base0 + sub] : 0.0f;
    int buf = 0, stage = 0;
    for (int64_t base = base0; base < p.M; base += stride) {
        const int64_t row = base + sub, ahead = row + stride;
        const float mean_next = ahead < p.M ? p.mean[ahead] : 0.0f, rstd_next = ahead < p.M ? p.rstd[ahead] : 0.0f;
        Piece<T, V> dyp[V == 1 ? C : 1], rp[V == 1 ? C : 1];
        if constexpr (S > 0) {
            fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
            cp_async_wait<S - 1>();
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = t + c * span;
                dyp[c].zero();
                rp[c].zero();
                if (row < p.M && k < pieces) {
                    dyp[c].load(p.dy + row * p.ld_dy + k);
                    rp[c].load(p.r + row * p.ld_r + k);
                }
            }
        }
        auto inputs = [&](int c, float (&dy)[V], float (&xhat)[V]) {
            Piece<T, V> a, b;
            if constexpr (S > 0) {
                a.raw = *slot(stage, 0, c);
                b.raw = *slot(stage, 1, c);
            } else {
                a = dyp[c];
                b = rp[c];
            }
            a.unpack(dy);
            b.unpack(xhat);
#pragma unroll
            for (int i = 0; i < V; ++i) xhat[i] = (xhat[i] - mean) * rstd;
        };
        auto weights = [&](int c, float (&v)[V]) {
            if constexpr (kHeld) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = w[c][i];
            } else {
                load_params<T, V>(p.w, static_cast<int64_t>(t + c * span) * V, v);
            }
        };
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (t + c * span >= pieces) continue;
            float dy[V], xhat[V], wc[V];
            inputs(c, dy, xhat);
            weights(c, wc);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gi = dy[i] * wc[i];
                c1 += gi;
                c2 = __fmaf_rn(gi, xhat[i], c2);
                dw[c][i] = __fmaf_rn(dy[i], xhat[i], dw[c][i]);
                db[c][i] += dy[i];
            }
        }
        const int width = MODE == NARROW ? team : 32;
        for (int o = width / 2; o; o >>= 1) {
            c1 += __shfl_xor_sync(0xFFFFFFFFu, c1, o);
            c2 += __shfl_xor_sync(0xFFFFFFFFu, c2, o);
        }
        if constexpr (MODE != NARROW) {
            // two buffers: a warp that runs ahead writes the other one, and cannot reach this one
            // again before every warp has passed the next row's barrier
            if (lane == 0) s_sum[buf][warp] = make_float2(c1, c2);
            __syncthreads();
            c1 = c2 = 0.0f;
            for (int k = 0; k < nw; ++k) {
                const float2 f = s_sum[buf][k];
                c1 += f.x;
                c2 += f.y;
            }
            buf ^= 1;
        }
        c1 *= inv_n;
        c2 *= inv_n;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t + c * span;
            if (row >= p.M || k >= pieces) continue;
            const int64_t j = static_cast<int64_t>(k) * V;
            float d[V], xhat[V], wc[V];
            inputs(c, d, xhat);
            weights(c, wc);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = rstd * (d[i] * wc[i] - c1 - xhat[i] * c2);
            if (p.dres) {
                Piece<T, V> a;
                if constexpr (S > 0) a.raw = *slot(stage, 2, c);
                else a.load(p.dres + row * p.ld_dres + k);
                a.unpack(xhat);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] += xhat[i];
            }
            Piece<T, V> out;
            out.pack(d);
            out.store(p.dx + row * p.ld_dx + j);
            if (p.dbranch) {
                if constexpr (DROP) {
                    uint32_t words[V];
                    words_at<V>(g, static_cast<uint32_t>(j), static_cast<uint32_t>(row), words);
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] = dropped(d[i], words[i], p.drop);
                    out.pack(d);
                }
                out.store(p.dbranch + row * p.ld_db + j);
            }
        }
        mean = mean_next;
        rstd = rstd_next;
        if constexpr (S > 0) stage = stage == S - 1 ? 0 : stage + 1;
    }
    pdl_launch_dependents();
    if constexpr (S > 0) cp_async_wait<0>();
    if (p.part == nullptr) return;

    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
    if constexpr (MODE == NARROW) {
        // lanes of the warp that took other rows of the same columns, then the warps in order
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i)
                for (int o = team; o < 32; o *= 2) {
                    dw[c][i] += __shfl_xor_sync(0xFFFFFFFFu, dw[c][i], o);
                    db[c][i] += __shfl_xor_sync(0xFFFFFFFFu, db[c][i], o);
                }
        const int n = static_cast<int>(p.N);
        for (int k = 0; k < nw; ++k) {
            if (warp == k && lane < team) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (t + c * span >= pieces) continue;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int j = (t + c * span) * V + i;
                        s_part[j] = k ? s_part[j] + dw[c][i] : dw[c][i];
                        s_part[n + j] = k ? s_part[n + j] + db[c][i] : db[c][i];
                    }
                }
            }
            __syncthreads();
        }
        for (int j = threadIdx.x; j < 2 * n; j += blockDim.x) part[j] = s_part[j];
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (t + c * span >= pieces) continue;
            const int64_t j = static_cast<int64_t>(t + c * span) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[j + i] = dw[c][i];
                part[p.N + j + i] = db[c][i];
            }
        }
    }
}

// Most partial rows of a call: CTAs of the row kernels that run at a time.
int parts_of(int64_t M, int64_t N) {
    const int64_t rows = N <= 1024 ? 4 : 1;  // rows that a CTA takes at a time, or so
    return static_cast<int>(std::min<int64_t>((M + rows - 1) / rows, std::min(1024, 4 * sm_count())));
}

template <typename T, int V, int C, RowsMode MODE, bool DROP>
cudaError_t launch_rows_as(BwdParams<T>& p, int team, unsigned block, cudaStream_t stream) {
    // one wave: as many CTAs as run at a time (the answer is kept per CTA size)
    static std::atomic<int> per_sm[33];
    const auto kern = ln_bwd_rows_kernel<T, V, C, MODE, DROP>;
    const size_t smem = size_t(ring_stages(V, C, MODE)) * 3 * C * block * 16;
    int n = per_sm[block / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 16 * 1024);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, static_cast<int>(block), smem);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
        per_sm[block / 32].store(n, std::memory_order_relaxed);
    }
    p.parts = std::min(p.parts, n * sm_count());
    return launch_pdl(kern, dim3(p.parts), dim3(block), smem, stream, p, team);
}

template <typename T, int V, int C, RowsMode MODE>
cudaError_t launch_rows(BwdParams<T>& p, int team, unsigned block, cudaStream_t stream) {
    return p.drop.on && p.dbranch ? launch_rows_as<T, V, C, MODE, true>(p, team, block, stream)
                                  : launch_rows_as<T, V, C, MODE, false>(p, team, block, stream);
}

// The one-pass kernels, where the row fits one; cudaErrorNotSupported where it
// does not.  Lowers p.parts to the partial rows that are written.
template <typename T, int V>
cudaError_t launch_bwd_rows(BwdParams<T>& p, cudaStream_t stream) {
    const int64_t pieces = p.N / V;
    constexpr int kMost = 16 / V;  // pieces of a thread of a CTA's row: 16 columns
    const auto threads = [&](int c) { return static_cast<unsigned>((pieces + 32 * c - 1) / (32 * c)) * 32; };
    if (pieces > 512 * kMost) {
        if constexpr (V > 1) {
            if (pieces <= 1024 * kMost) return launch_rows<T, V, kMost, BROAD>(p, 0, threads(kMost), stream);
        }
        return cudaErrorNotSupported;
    }
    if (pieces > 128) {
        if (pieces <= 256 * (kMost / 2)) return launch_rows<T, V, kMost / 2, WIDE>(p, 0, threads(kMost / 2), stream);
        return launch_rows<T, V, kMost, WIDE>(p, 0, threads(kMost), stream);
    }
    int team = 1;
    while (team < 32 && team < pieces) team *= 2;
    switch ((pieces + team - 1) / team) {
        case 1: return launch_rows<T, V, 1, NARROW>(p, team, 128, stream);
        case 2: return launch_rows<T, V, 2, NARROW>(p, team, 128, stream);
        case 3: return launch_rows<T, V, 3, NARROW>(p, team, 128, stream);
        default: return launch_rows<T, V, 4, NARROW>(p, team, 128, stream);
    }
}

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
    p.w = Params<T>{a.weight, a.param_dtype == FP8Q_FP32, 1.0f};
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
    constexpr int V = 16 / sizeof(T);
    const bool pieces = a.N % V == 0 && rows16(a.dy, a.ld_dy, sizeof(T)) && rows16(a.r, a.ld_r, sizeof(T)) &&
                        rows16(a.dresidual, a.ld_dresidual, sizeof(T)) && rows16(a.dx, a.ld_dx, sizeof(T)) &&
                        rows16(a.dbranch, a.ld_dbranch, sizeof(T)) && aligned16(a.weight);
    cudaError_t e = pieces ? launch_bwd_rows<T, V>(p, stream) : launch_bwd_rows<T, 1>(p, stream);
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
    if (cols && e == cudaSuccess)
        e = launch_pdl(ln_bwd_reduce_kernel, dim3(static_cast<unsigned>((2 * a.N + 31) / 32)), dim3(1024), 0, stream,
                       static_cast<const float*>(p.part), p.parts, a.N, a.dweight, a.dbias,
                       (a.flags & FP8Q_ACCUMULATE) != 0);
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
