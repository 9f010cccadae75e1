// block_norm.cuh -- the one-pass kernels of block_norm_fwd and block_norm_bwd, which
// block_norm.cu launches; each element type, on and off the 16-byte grid, is a
// translation unit of its own (block_norm_*.cu), so that they compile side by side.
#pragma once

#include "common.cuh"
#include "norm_ops.cuh"

#include <algorithm>

namespace fp8q {

template <typename T>
struct BnFwd {
    int64_t M, N;
    const T* x;
    int64_t ldx;
    const T* res;
    int64_t ld_res;
    T* r_out;
    int64_t ld_r;
    T* y;
    int64_t ldy;
    Params<T> w, wp;       // of the norm before the next block; of the block's output
    const float* gate;     // [M] or NULL
    const float* alpha;    // or NULL: 1
    float* rstd;
    float* rstd_post;
    float eps;
    bool post, pre;        // norm after the block, norm before the next one
    bool alone;            // one CTA, whose maximum and count are the call's: stored, not added
    QuantOut quant;
};

template <typename T>
struct BnBwd {
    int64_t M, N;
    const T* dy;           // NULL: no norm before the next block
    int64_t ld_dy;
    const T* r;
    int64_t ld_r;
    const T* dr;           // the stream's gradient on its other way, or NULL
    int64_t ld_dr;
    const T* x;            // NULL: nothing of the block's output is wanted
    int64_t ldx;
    const T* res;          // NULL unless dalpha is wanted
    int64_t ld_res;
    T* dres;
    int64_t ld_dres;
    T* dx;
    int64_t ld_dx;
    Params<T> w, wp;
    const float* gate;
    const float* alpha;
    const float* rstd;
    const float* rstd_post;
    float* dgate;
    float* part;           // [parts][2][N] sums of dw and dwp, then [parts] of dalpha; NULL: not wanted
    int parts;
    bool post;
};

namespace {

__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// (a0, a1) -> a0 + a1
__device__ __forceinline__ float fold(f32x2 v) {
    const float2 f = split(v);
    return f.x + f.y;
}

// The maximum and count of a call's only CTA: stored, so that nothing has to clear them first.
__device__ __forceinline__ void store_quant(const QuantOut& o, uint32_t amax, uint32_t nsat) {
    __shared__ uint32_t s_amax[16], s_sat[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    nsat = __reduce_add_sync(0xFFFFFFFFu, nsat);
    if (lane == 0) {
        s_amax[warp] = amax;
        s_sat[warp] = nsat;
    }
    __syncthreads();
    if (warp != 0) return;
    amax = __reduce_max_sync(0xFFFFFFFFu, lane < nw ? s_amax[lane] : 0u);
    nsat = __reduce_add_sync(0xFFFFFFFFu, lane < nw ? s_sat[lane] : 0u);
    if (lane != 0) return;
    if (o.amax) *o.amax = __uint_as_float(amax);
    if (o.sat) *o.sat = nsat;
}
template <typename T>
__device__ __forceinline__ void finish_quant(const BnFwd<T>& p, uint32_t amax, uint32_t nsat) {
    if (!p.quant.on) return;
    if (p.alone) store_quant(p.quant, amax, nsat);
    else publish_quant(p.quant, amax, nsat);
}

// cp.async of the first `bytes` bytes of a granule, and zeros for the others.
__device__ __forceinline__ void cp_async16_part(uint32_t smem_addr, const void* gmem, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(smem_addr), "l"(gmem), "r"(bytes) : "memory");
}

// A thread's columns.  On the 16-byte grid a thread has whole 16-byte pieces: piece t + 32 c
// of its row, c < C, V columns each.  Off it (SHIFT) neither rows nor tensors of one row share an
// alignment, and a thread has the 4-byte words of its range of columns that lie L lanes apart: pairs
// of adjacent 2-byte columns, or single 4-byte ones.  The ring then holds the 16-byte granules that
// a row touches, one after the other, and a word is cut from the two that it may lie across by one
// funnel shift; reads are free of bank conflicts and stores whole words, shifted by one element
// through the neighbouring lane where the row starts between two words.  The row's last granule is copied
// in part and the rest zero-filled, so that nothing read needs a check.  (Cutting whole pieces from two
// granules each, and joining them for the stores: forward bf16 65536 x 1601 315 us, backward 451;
// now 222 and 366.)
// BRANCH: rows that start on a word are told from the others by a branch (forward bf16 65536 x 1601
// 277 us without, 222 with; the backward, short of registers, 389 without and 437 with).
template <typename T, int C, bool SHIFT, bool BRANCH>
struct Columns {
    static constexpr int V = 16 / sizeof(T), H = V / 2;
    int t, lanes, first, N;  // lane of the range, its lanes, its first column
    // pair i of piece c: its first column, and how far its second one is
    __device__ __forceinline__ int col(int c, int i) const {
        if constexpr (!SHIFT) return first + (t + 32 * c) * V + 2 * i;
        else if constexpr (sizeof(T) == 2) return first + 2 * (t + lanes * (c * H + i));
        else return first + t + lanes * 2 * (c * H + i);
    }
    __device__ __forceinline__ int apart() const { return SHIFT && sizeof(T) == 4 ? lanes : 1; }
    // whether the thread's piece c has columns of the row (on the grid: all or none of them)
    __device__ __forceinline__ bool has(int c) const { return col(c, 0) < N; }
    __device__ __forceinline__ bool has(int c, int i, int e) const { return col(c, i) + e * apart() < N; }

    // The parameters of pieces c0 .. c0 + P - 1 (0 behind the row): every load is under way before the
    // first is used.
    template <int P>
    __device__ __forceinline__ void params(const Params<T>& w, int c0, f32x2 (&v)[P][H]) const {
        const float* const f = static_cast<const float*>(w.p);
        const T* const h = static_cast<const T*>(w.p);
        if (w.p == nullptr) {
#pragma unroll
            for (int k = 0; k < P * H; ++k)
                v[k / H][k % H] = pair_of(has(c0 + k / H, k % H, 0) ? w.none : 0.0f, has(c0 + k / H, k % H, 1) ? w.none : 0.0f);
        } else if constexpr (!SHIFT) {  // (whole pieces of aligned vectors)
            if (w.f32) {
                float4 raw[P][V / 4];
#pragma unroll
                for (int k = 0; k < P * (V / 4); ++k) {
                    const int c = k / (V / 4), i = k % (V / 4);
                    raw[c][i] = has(c0 + c) ? __ldg(reinterpret_cast<const float4*>(f + col(c0 + c, 2 * i))) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
                for (int k = 0; k < P * (V / 4); ++k) {
                    const float4 q = raw[k / (V / 4)][k % (V / 4)];
                    v[k / (V / 4)][2 * (k % (V / 4))] = pair_of(q.x, q.y);
                    v[k / (V / 4)][2 * (k % (V / 4)) + 1] = pair_of(q.z, q.w);
                }
            } else {
                Piece<T, V> raw[P];
#pragma unroll
                for (int c = 0; c < P; ++c)
                    raw[c].raw = has(c0 + c) ? __ldg(reinterpret_cast<const uint4*>(h + col(c0 + c, 0))) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < P; ++c) unpack2(raw[c], v[c]);
            }
        } else if (w.f32) {
            float raw[P * H][2];
#pragma unroll
            for (int k = 0; k < P * H; ++k) {
                const int c = c0 + k / H, i = k % H, j = col(c, i);
                raw[k][0] = has(c, i, 0) ? __ldg(f + j) : 0.0f;
                raw[k][1] = has(c, i, 1) ? __ldg(f + j + apart()) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < P * H; ++k) v[k / H][k % H] = pair_of(raw[k][0], raw[k][1]);
        } else {
            T raw[P * H][2];
            const T zero = from_f32<T>(0.0f);
#pragma unroll
            for (int k = 0; k < P * H; ++k) {
                const int c = c0 + k / H, i = k % H, j = col(c, i);
                raw[k][0] = has(c, i, 0) ? h[j] : zero;
                raw[k][1] = has(c, i, 1) ? h[j + apart()] : zero;
            }
#pragma unroll
            for (int k = 0; k < P * H; ++k) v[k / H][k % H] = pair_of(to_f32(raw[k][0]), to_f32(raw[k][1]));
        }
    }
    // The copies of this thread of one row of a tensor into its range's slots at `to`.
    __device__ __forceinline__ void fill(uint32_t to, const T* row) const {
        if constexpr (SHIFT) {
            const uint32_t mis = granule_offset(row);
            const uint8_t* base = reinterpret_cast<const uint8_t*>(row) - mis;
            const int begin = first * static_cast<int>(sizeof(T)), end = N * static_cast<int>(sizeof(T)) + static_cast<int>(mis);
#pragma unroll
            for (int c = 0; c <= C; ++c) {
                const int g = c < C ? t + lanes * c : lanes * C, at = begin + g * 16;
                // (what lies behind the row is zeros in the slots: its last granule is copied in part)
                const int bytes = min(max(end - at, 0), 16);
                if (c < C || t == lanes - 1) cp_async16_part(to + g * 16, bytes > 0 ? base + at : base, bytes);
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (has(c)) cp_async16(to + (t + 32 * c) * 16, row + col(c, 0));
        }
    }
    // Whether the range ends behind the row (the same for all lanes).
    __device__ __forceinline__ bool cut() const { return first + lanes * C * V > N; }
    __device__ __forceinline__ static f32x2 unpack_word(uint32_t u) {
        if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
            return pair_of(f.x, f.y);
        } else {
            return pair_of(bf16lo_to_f32(u), bf16hi_to_f32(u));
        }
    }
    // Columns behind the row: 0.
    __device__ __forceinline__ void clip(int c, f32x2 (&v)[H]) const {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 f = split(v[i]);
            v[i] = pair_of(has(c, i, 0) ? f.x : 0.0f, has(c, i, 1) ? f.y : 0.0f);
        }
    }
    // Piece c from the slots; `row` for its alignment.  Columns behind the row are zeros.
    __device__ __forceinline__ void read(const uint4* slots, const T* row, int c, f32x2 (&v)[H]) const {
        if constexpr (SHIFT) {
            const uint32_t mis = granule_offset(row);
            const uint32_t* const words = reinterpret_cast<const uint32_t*>(slots) + (mis >> 2) + t;
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const uint32_t* w = words + lanes * 2 * (c * H + i);
                    v[i] = pair_of(__uint_as_float(w[0]), __uint_as_float(w[lanes]));
                }
            } else if (!BRANCH || (mis & 2)) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const uint32_t* w = words + lanes * (c * H + i);
                    v[i] = unpack_word(__funnelshift_r(w[0], w[1], (mis & 2) * 8));
                }
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = unpack_word(words[lanes * (c * H + i)]);
            }
        } else {
            Piece<T, V> a;
            a.raw = slots[t + 32 * c];
            unpack2(a, v);
        }
    }
    // Piece c, already rounded, to the row; `carry` goes from piece to piece.  All lanes call it; `in`: the
    // row exists; tail: the piece may end behind the row (always, where teams of lanes have rows of their own).
    __device__ __forceinline__ void put(T* row, int c, uint4 q, uint32_t& carry, bool in, bool tail) const {
        if constexpr (!SHIFT) {
            if (in && has(c)) st_v4(row + col(c, 0), q);
            return;
        }
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
        if constexpr (sizeof(T) == 4) {
            uint32_t* const out = reinterpret_cast<uint32_t*>(row);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (in && (!tail || has(c, i / 2, i & 1))) out[col(c, i / 2) + (i & 1) * lanes] = u[i];
        } else {
            uint16_t* const out = reinterpret_cast<uint16_t*>(row);
            const bool between = reinterpret_cast<uintptr_t>(row) & 2;  // the row starts between two words
            const int rest = N - first - 2 * t;
            if (C > 1 && !between) {  // (a warp's lanes have one row: all or none of them)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int left = !in ? -1 : tail ? rest - 2 * lanes * (c * H + i) : 2;
                    if (left >= 2) *reinterpret_cast<uint32_t*>(out + col(c, i)) = u[i];
                    else if (left == 1) out[col(c, i)] = static_cast<uint16_t>(u[i]);
                }
                return;
            }
            const int lane = threadIdx.x & 31, from = (lane & ~(lanes - 1)) | ((t + lanes - 1) & (lanes - 1));
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int j = col(c, i), left = !in ? -1 : tail ? rest - 2 * lanes * (c * H + i) : 2;  // columns from this pair's first on
                const uint32_t before = __shfl_sync(0xFFFFFFFFu, u[i], from);
                if (!between) {
                    if (left >= 2) *reinterpret_cast<uint32_t*>(out + j) = u[i];
                    else if (left == 1) out[j] = static_cast<uint16_t>(u[i]);
                } else {
                    const uint32_t prev = t == 0 ? carry : before;
                    const bool head = c == 0 && i == 0 && t == 0, last = c == C - 1 && i == H - 1 && t == lanes - 1;
                    if (left >= 1) {
                        if (head) out[j] = static_cast<uint16_t>(u[i]);
                        else *reinterpret_cast<uint32_t*>(out + j - 1) = __funnelshift_r(prev, u[i], 16);
                        if (last && left >= 2) out[j + 1] = static_cast<uint16_t>(u[i] >> 16);
                    } else if (left == 0 && !head) {
                        out[j - 1] = static_cast<uint16_t>(prev >> 16);
                    }
                }
                carry = before;  // lane 0's: the range's last lane
            }
        }
    }
    // The codes of piece c of the rounded y, its magnitudes and saturations.
    __device__ __forceinline__ void quant(const QuantOut& o, float s, uint8_t* row, int c, bool tail, const Piece<T, V>& y,
                                          uint32_t& amax, uint32_t& amax2, uint32_t& nsat) const {
        if constexpr (SHIFT) {
            float f[V];
            y.unpack(f);
            const float fmax = fp8_max_value(o.fmt);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float v0 = __fmul_rn(f[2 * i], s), v1 = __fmul_rn(f[2 * i + 1], s);
                const int j = col(c, i), k = j + apart();
                const uint32_t q = cast_pair(v0, v1, o.fmt);
                if (!tail || j < N) {
                    amax = max(amax, __float_as_uint(fabsf(f[2 * i])));
                    nsat += fabsf(v0) > fmax;
                    if (row) row[j] = static_cast<uint8_t>(q);
                }
                if (!tail || k < N) {
                    amax = max(amax, __float_as_uint(fabsf(f[2 * i + 1])));
                    nsat += fabsf(v1) > fmax;
                    if (row) row[k] = static_cast<uint8_t>(q >> 8);
                }
            }
        } else {
            uint8_t* dst = row ? row + col(c, 0) : nullptr;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                if (o.fmt == FP8Q_E5M2) quant_bf16x8<FP8Q_E5M2>(s, y.raw, dst, amax2, nsat);
                else quant_bf16x8<FP8Q_E4M3>(s, y.raw, dst, amax2, nsat);
            } else {
                quant_piece<T, V>(o, s, y, dst, V, true, amax, nsat);
            }
        }
    }
};

// Slots of a warp's ring for one row of one tensor; rows: each team of lanes has a row of its own.
__host__ __device__ constexpr int bn_slots(int C, bool shift, bool rows) { return !shift ? 32 * C : rows ? 64 : 32 * C + 1; }

// The forward: one pass over rows, from a ring of S rows in shared memory.
//   NARROW (CTA = false)  `team` lanes of a warp take a row, up to 64 columns a lane
//   CTA                   a CTA of up to 512 threads takes a row, 32 columns a thread
// The row stays in registers from its one read to its one write; its two sums of squares (of
// the block's output, and of the stored stream) are team shuffles, or an exchange each.
// Weights: in registers up to 32 columns a lane, in shared memory above.
// What bounds it: memory on the 16-byte grid (bf16 131072 x 1600 with codes 302 to 316 us, 0.92 to 0.88 of the
// measured copy rate; 65536 x 768 69 us, 0.86; 8192 x 16384 160 to 180 us, 0.99 to 0.88); off it memory for
// float32 (65536 x 1001 175 us, 0.88) and the words' instructions for bf16 (65536 x 1601 222 us, 0.56; narrow rows
// also leave lanes of their last piece idle, and codes go byte by byte: 333 columns 55 us, 0.47, with codes 70,
// 0.42, 99 columns 24 us, 0.32); for one row the launch.
template <typename T, int C, bool CTA, bool SHIFT, int S>
__global__ void __launch_bounds__(CTA ? 512 : 128)
bn_fwd_kernel(const BnFwd<T> p, int team) {
    extern __shared__ uint4 s_ring[];
    __shared__ float s_sum[2][2][16];
    constexpr int V = 16 / sizeof(T), H = V / 2;
    constexpr bool kHeld = C * V <= 32;
    constexpr int kTensor = bn_slots(C, SHIFT, !CTA && C == 1), kStage = 2 * kTensor;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if constexpr (C > 1 || CTA) team = 32;
    const int N = static_cast<int>(p.N);
    const Columns<T, C, SHIFT, true> my{lane & (team - 1), team, CTA ? warp * 32 * C * V : 0, N};
    const float inv_n = 1.0f / static_cast<float>(N);
    const f32x2 zero2 = pair_of(0.0f, 0.0f);
    uint32_t carry = 0;
    pdl_wait();

    const float s = p.quant.on ? *p.quant.scale : 0.0f;
    const float alpha = p.alpha ? *p.alpha : 1.0f;
    uint32_t amax = 0, amax2 = 0, nsat = 0;

    const int rows_warp = CTA ? 1 : 32 / team, rows_cta = CTA ? 1 : rows_warp * nw;
    const uint32_t M = static_cast<uint32_t>(p.M), stride = gridDim.x * rows_cta, base0 = blockIdx.x * rows_cta;
    const uint32_t sub = CTA ? 0 : warp * rows_warp + lane / team;
    // [stage][x, residual][slots], a team's from its own first slot
    uint4* const ring = s_ring + warp * (S * kStage) + (lane / team) * (team * C + (SHIFT ? 1 : 0));
    const uint32_t ring_at = smem_u32(ring);
    // (off the grid a range's last columns may lie behind the row; on it a piece has all or none)
    const bool cut = SHIFT && my.cut();
    auto tail = [&](int c) { return SHIFT && (CTA ? cut : c == C - 1); };
    auto fill = [&](int stage, uint32_t row) {  // nothing for a row past the last
        if (row < M) {
            const uint32_t to = ring_at + stage * kStage * 16;
            my.fill(to, p.x + row * p.ldx);
            if (p.res) my.fill(to + kTensor * 16, p.res + row * p.ld_res);
        }
        cp_async_commit();
    };
    if constexpr (!SHIFT) {  // pieces past the row are zeros in every stage, and stay so
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (!my.has(c))
                for (int k = 0; k < S * 2; ++k) ring[k * kTensor + my.t + 32 * c] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);

    // [w, wp][four columns of a piece][c][lane]
    float4* const s_par = reinterpret_cast<float4*>(s_ring + nw * (S * kStage)) + lane;
    f32x2 w[kHeld ? C : 1][H], wp[kHeld ? C : 1][H];
    if constexpr (kHeld) {
        my.params(p.w, 0, w);
        my.params(p.wp, 0, wp);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (warp != c % 4) continue;
            f32x2 f[2][1][H];
            my.params(p.w, c, f[0]);
            my.params(p.wp, c, f[1]);
#pragma unroll
            for (int k = 0; k < 2 * (V / 4); ++k) {
                const int q = k / (V / 4), i = k % (V / 4);
                const float2 a = split(f[q][0][2 * i]), b = split(f[q][0][2 * i + 1]);
                s_par[(k * C + c) * 32] = make_float4(a.x, a.y, b.x, b.y);
            }
        }
        __syncthreads();
    }
    auto weights = [&](int q, int c, f32x2 (&f)[H]) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < H; ++i) f[i] = q ? wp[c][i] : w[c][i];
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 v = s_par[((q * (V / 4) + i) * C + c) * 32];
                f[2 * i] = pair_of(v.x, v.y);
                f[2 * i + 1] = pair_of(v.z, v.w);
            }
        }
    };

    auto row_sum = [&](float v, float* sums) {  // in a fixed order
        v = team_sum<C == 1 && !CTA>(v, team);
        if constexpr (CTA) {
            if (lane == 0) sums[warp] = v;
            __syncthreads();
            v = 0.0f;
            for (int k = 0; k < nw; ++k) v += sums[k];
        }
        return v;
    };
    float gate_next = 1.0f;  // read a row ahead
    if (p.gate && base0 + sub < M) gate_next = p.gate[base0 + sub];
    int stage = 0, buf = 0;
    for (uint32_t base = base0; base < M; base += stride) {
        const uint32_t row = base + sub;
        const bool in = row < M;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        const float gate = gate_next;
        if (p.gate && row + stride < M) gate_next = p.gate[row + stride];
        cp_async_wait<S - 1>();
        if constexpr (SHIFT) __syncwarp();
        const uint4* at = ring + stage * kStage;
        const T* const x_row = p.x + row * p.ldx;
        const T* const res_row = p.res + row * p.ld_res;
        f32x2 v[C][H];
        f32x2 sq[2] = {zero2, zero2};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            my.read(at, x_row, c, v[c]);
#pragma unroll
            for (int i = 0; i < H; ++i) sq[i & 1] = fma2(v[c][i], v[c][i], sq[i & 1]);
        }
        float rp = 1.0f;
        if (p.post) {
            const float sum = row_sum(fold(add2(sq[0], sq[1])), s_sum[buf][0]);
            rp = 1.0f / sqrtf(__fmaf_rn(sum, inv_n, p.eps));
            if (p.rstd_post && in && my.t + my.first == 0) p.rstd_post[row] = rp;
        }
        const f32x2 rp2 = pair_of(rp, rp), gate2 = pair_of(gate, gate), alpha2 = pair_of(alpha, alpha);
        sq[0] = sq[1] = zero2;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            f32x2 f[H];
            weights(1, c, f);
#pragma unroll
            for (int i = 0; i < H; ++i) v[c][i] = mul2(mul2(mul2(v[c][i], rp2), f[i]), gate2);
            if (p.res) {
                f32x2 r[H];
                my.read(at + kTensor, res_row, c, r);
#pragma unroll
                for (int i = 0; i < H; ++i) v[c][i] = fma2(alpha2, r[i], v[c][i]);
            }
            Piece<T, V> a;
            pack2(a, v[c]);
            if (p.r_out) my.put(p.r_out + row * p.ld_r, c, a.raw, carry, in, tail(c));
            unpack2(a, v[c]);
            // (behind the row an infinite gate or alpha times the zeros there is NaN)
            if constexpr (SHIFT) {
                if (tail(c)) my.clip(c, v[c]);
            } else if (!my.has(c)) {
#pragma unroll
                for (int i = 0; i < H; ++i) v[c][i] = zero2;
            }
#pragma unroll
            for (int i = 0; i < H; ++i) sq[i & 1] = fma2(v[c][i], v[c][i], sq[i & 1]);
        }
        if (p.pre) {
            const float sum = row_sum(fold(add2(sq[0], sq[1])), s_sum[buf][1]);
            const float rstd = 1.0f / sqrtf(__fmaf_rn(sum, inv_n, p.eps));
            if (p.rstd && in && my.t + my.first == 0) p.rstd[row] = rstd;
            const f32x2 rstd2 = pair_of(rstd, rstd);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!SHIFT && !(in && my.has(c))) continue;
                f32x2 f[H];
                weights(0, c, f);
#pragma unroll
                for (int i = 0; i < H; ++i) v[c][i] = mul2(mul2(v[c][i], rstd2), f[i]);
                Piece<T, V> y;
                pack2(y, v[c]);
                if (p.y) my.put(p.y + row * p.ldy, c, y.raw, carry, in, tail(c));
                if (p.quant.on && in) my.quant(p.quant, s, p.quant.q ? p.quant.q + row * p.N : nullptr, c, tail(c), y, amax, amax2, nsat);
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        buf ^= 1;
        if constexpr (SHIFT) __syncwarp();  // the granules that other lanes read may be overwritten now
    }
    pdl_launch_dependents();
    cp_async_wait<0>();
    finish_quant(p, max(amax, max16x2(amax2) << 16), nsat);
}

template <typename T, int C, bool CTA, bool SHIFT, int S = 3>
cudaError_t launch_bn_fwd_as(const BnFwd<T>& p, int team, unsigned block, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    static DeviceTable<17> table;
    const auto kern = bn_fwd_kernel<T, C, CTA, SHIFT, S>;
    size_t smem = size_t(S) * 2 * (block / 32) * bn_slots(C, SHIFT, !CTA && C == 1) * 16;
    if (C * V > 32) smem += size_t(2) * C * 32 * V * sizeof(float);
    int n = 0;
    const cudaError_t e = resident_ctas(table, kern, block, smem, kMaxRing, &n);
    if (e != cudaSuccess) return e;
    const int64_t rows = CTA ? 1 : 128 / team;
    const int64_t grid = std::min<int64_t>((p.M + rows - 1) / rows, int64_t(n) * sm_count());
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, p, team);
}

// The backward.  A thread keeps its columns' weights and sums for all its rows.
//   NARROW   `team` lanes of a warp take a row, up to 3 pieces a lane
//   WIDE     a group of `team` warps takes a row; a CTA is several groups
//   CLUSTER  the CTAs of a cluster take a row, all their warps one group; sums cross by
//            distributed shared memory
//     rhat = r rstd, g = dy w;  dr = dr_in + rstd (g - rhat sum(g rhat) / N)
//     xhat = x rstd_post;       e = sum(dr wp xhat)
//     dx = gate rstd_post (dr wp - xhat e / N)  [post],  gate dr wp  [not post]
// The row's inputs come through a ring of rows in shared memory: three, or two where the
// residual is read too.
// What bounds it: memory where the rows are on the grid and fill the lanes (bf16 65536 x 2048 239 us,
// 1.00 of the measured copy rate; 131072 x 1600 400 us, 0.93; fp32 65536 x 1600 355 us, 1.04); off it the
// instructions that cut words and shift them back (bf16 65536 x 1601 366 us, 0.51; fp32, which has none to cut,
// 65536 x 1001 240 us, 0.97; bf16 333 columns 79 us, 0.49, 99 columns 39 us, 0.30); rows over a cluster (8192 x 16384
// 419 us, 0.57; 12288 columns 383, 0.46; float32 8192 columns 382, 0.62, off the grid 16384 x 5001 738, 0.39) wait
// at the cluster's barriers for the stores before them.
enum BnMode { BN_NARROW, BN_WIDE, BN_CLUSTER };
constexpr int bn_bwd_stages(bool alpha) { return alpha ? 2 : 3; }
enum { IN_DY, IN_R, IN_DR, IN_X, IN_RES };

template <typename T, int C, BnMode MODE, bool ALPHA, bool SHIFT>
__global__ void __launch_bounds__(C >= 3 ? 256 : 512, 1)
bn_bwd_kernel(const BnBwd<T> p, int team) {
    extern __shared__ uint4 s_ring[];
    __shared__ float s_sum[2][2][16];
    // dalpha's by warp: cells of their own, since a CTA of the cluster that is late may still read its last row's
    // sum from s_sum (nothing orders that before this CTA's end where a row has one sum).  32 of them, so that the
    // ring behind starts on a 128-byte line (off one, 8192 x 16384 499 us, on it 459).
    __shared__ float s_alpha[ALPHA ? 32 : 1];
    constexpr int V = 16 / sizeof(T), H = V / 2, S = bn_bwd_stages(ALPHA), TENSORS = ALPHA ? 5 : 4;
    constexpr bool kWarp = MODE == BN_NARROW;
    constexpr int kTensor = bn_slots(C, SHIFT, kWarp && C == 1), kStage = TENSORS * kTensor;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const uint32_t rank = MODE == BN_CLUSTER ? cluster_ctarank() : 0, ctas = MODE == BN_CLUSTER ? cluster_nctarank() : 1;
    if constexpr (MODE == BN_CLUSTER) team = nw;
    // otherwise (NARROW) team = lanes of a row
    const int group = kWarp ? warp : warp / team, wg = kWarp ? 0 : rank * nw + warp - group * team;
    const int lanes = !kWarp || C > 1 ? 32 : team;
    const int N = static_cast<int>(p.N);
    const Columns<T, C, SHIFT, false> my{lane & (lanes - 1), lanes, wg * 32 * C * V, N};
    const bool leads = my.t + my.first == 0;
    const float inv_n = 1.0f / static_cast<float>(N);
    const f32x2 zero2 = pair_of(0.0f, 0.0f);
    uint32_t carry = 0;
    pdl_wait();
    const float alpha = p.alpha ? *p.alpha : 1.0f;
    f32x2 dalpha2 = zero2;

    const int groups = kWarp ? nw : nw / team, rows_warp = kWarp ? 32 / lanes : 1, rows_cta = groups * rows_warp;
    const uint32_t M = static_cast<uint32_t>(p.M), block = blockIdx.x / ctas;
    const uint32_t stride = gridDim.x / ctas * rows_cta, base0 = block * rows_cta;
    const uint32_t sub = group * rows_warp + (kWarp ? lane / lanes : 0);
    uint4* const ring = s_ring + warp * (S * kStage) + (lane / lanes) * (lanes * C + (SHIFT ? 1 : 0));
    const uint32_t ring_at = smem_u32(ring);
    auto tail = [&](int c) { return SHIFT && (!kWarp || c == C - 1); };
    auto fill_tensor = [&](uint32_t to, const T* base, int64_t at) {
        if (base) my.fill(to, base + at);
    };
    auto fill = [&](int stage, uint32_t row) {
        if (row < M) {
            const uint32_t to = ring_at + stage * kStage * 16, step = kTensor * 16;
            fill_tensor(to + IN_DY * step, p.dy, row * p.ld_dy);
            fill_tensor(to + IN_R * step, p.r, row * p.ld_r);
            fill_tensor(to + IN_DR * step, p.dr, row * p.ld_dr);
            fill_tensor(to + IN_X * step, p.x, row * p.ldx);
            if constexpr (ALPHA) fill_tensor(to + IN_RES * step, p.res, row * p.ld_res);
        }
        cp_async_commit();
    };
    if constexpr (!SHIFT) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (!my.has(c))
                for (int k = 0; k < S * TENSORS; ++k) ring[k * kTensor + my.t + 32 * c] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fill(k, base0 + sub + k * stride);

    f32x2 w[C][H], wp[C][H], dw[C][H], dwp[C][H];
    my.params(p.w, 0, w);
    my.params(p.wp, 0, wp);
#pragma unroll
    for (int k = 0; k < C * H; ++k) dw[k / H][k % H] = dwp[k / H][k % H] = zero2;

    auto group_sum = [&](float v, float* sums) {  // in a fixed order
        v = team_sum<C == 1 && kWarp>(v, lanes);
        if constexpr (MODE == BN_WIDE) {
            if (lane == 0) sums[warp] = v;
            named_barrier(1 + group, team * 32);
            v = 0.0f;
            for (int k = 0; k < team; ++k) v += sums[group * team + k];
        }
        if constexpr (MODE == BN_CLUSTER) {
            if (lane == 0) sums[warp] = v;
            cluster_sync_all();
            // lane k adds warp k of every CTA, then the lanes are added
            v = 0.0f;
            if (lane < nw)
                for (uint32_t r = 0; r < ctas; ++r) v += ld_cluster_f32(mapa_shared(smem_u32(sums + lane), r));
            v = team_sum<false>(v, 32);
        }
        return v;
    };
    // a row's gate and statistics, read a row ahead
    float gate_next = 1.0f, rp_next = 1.0f, rs_next = 0.0f;
    auto scalars = [&](uint32_t row) {
        if (row >= M) return;
        if (p.gate) gate_next = p.gate[row];
        if (p.rstd_post) rp_next = p.rstd_post[row];
        if (p.dy) rs_next = p.rstd[row];
    };
    scalars(base0 + sub);
    int stage = 0, buf = 0;
    // (a group, or a warp with one row, is done at its own last row; lanes of several rows together)
    for (uint32_t base = base0; (!kWarp || C > 1 ? base + sub : base) < M; base += stride) {
        const uint32_t row = base + sub;
        const bool in = row < M;
        fill(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * stride);
        const float gate = gate_next, rp = rp_next, rs = rs_next;
        scalars(row + stride);
        cp_async_wait<S - 1>();
        if constexpr (SHIFT) __syncwarp();
        const uint4* at = ring + stage * kStage;
        auto read = [&](int which, const T* base_p, int64_t off, int c, f32x2 (&v)[H]) {
            if (base_p == nullptr) {
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = zero2;
                return;
            }
            my.read(at + which * kTensor, base_p + off, c, v);
        };
        f32x2 dr[C][H];
        // the norm before the next block
        if (p.dy) {
            const f32x2 rs2 = pair_of(rs, rs);
            f32x2 rhat[C][H], acc[2] = {zero2, zero2};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 dy[H];
                read(IN_DY, p.dy, row * p.ld_dy, c, dy);
                read(IN_R, p.r, row * p.ld_r, c, rhat[c]);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    rhat[c][i] = mul2(rhat[c][i], rs2);
                    if (in) dw[c][i] = fma2(dy[i], rhat[c][i], dw[c][i]);
                    dr[c][i] = mul2(dy[i], w[c][i]);
                    acc[i & 1] = fma2(dr[c][i], rhat[c][i], acc[i & 1]);
                }
            }
            const float along = -group_sum(fold(add2(acc[0], acc[1])), s_sum[buf][0]) * inv_n;
            const f32x2 along2 = pair_of(along, along);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 d[H];
                read(IN_DR, p.dr, row * p.ld_dr, c, d);
#pragma unroll
                for (int i = 0; i < H; ++i) dr[c][i] = fma2(fma2(rhat[c][i], along2, dr[c][i]), rs2, d[i]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) read(IN_DR, p.dr, row * p.ld_dr, c, dr[c]);
        }
        if constexpr (ALPHA) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 f[H];
                read(IN_RES, p.res, row * p.ld_res, c, f);
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (in) dalpha2 = fma2(dr[c][i], f[i], dalpha2);
            }
        }
        if (p.dres) {
            const f32x2 alpha2 = pair_of(alpha, alpha);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                f32x2 f[H];
#pragma unroll
                for (int i = 0; i < H; ++i) f[i] = mul2(dr[c][i], alpha2);
                Piece<T, V> a;
                pack2(a, f);
                my.put(p.dres + row * p.ld_dres, c, a.raw, carry, in, tail(c));
            }
        }
        // the block's output, its norm and its gate
        if (p.x) {
            const f32x2 rp2 = pair_of(rp, rp), gate2 = pair_of(gate, gate);
            f32x2 xhat[C][H], acc[2] = {zero2, zero2};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                read(IN_X, p.x, row * p.ldx, c, xhat[c]);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    xhat[c][i] = mul2(xhat[c][i], rp2);
                    if (in) dwp[c][i] = fma2(mul2(dr[c][i], gate2), xhat[c][i], dwp[c][i]);
                    dr[c][i] = mul2(dr[c][i], wp[c][i]);
                    acc[i & 1] = fma2(dr[c][i], xhat[c][i], acc[i & 1]);
                }
            }
            float along = 0.0f;
            if (p.post || p.dgate) {
                along = group_sum(fold(add2(acc[0], acc[1])), s_sum[buf][1]);
                if (p.dgate && in && leads) p.dgate[row] = along;
            }
            if (p.dx) {
                const float a1 = p.post ? -along * inv_n : 0.0f;
                const f32x2 along2 = pair_of(a1, a1);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    f32x2 f[H];
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        f[i] = p.post ? mul2(fma2(xhat[c][i], along2, dr[c][i]), rp2) : dr[c][i];
                        f[i] = mul2(f[i], gate2);
                    }
                    Piece<T, V> a;
                    pack2(a, f);
                    my.put(p.dx + row * p.ld_dx, c, a.raw, carry, in, tail(c));
                }
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        buf ^= 1;
        if constexpr (SHIFT) __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
    pdl_launch_dependents();
    if (p.part) {
        // the CTA's sums in shared memory: [warp or group][dw, dwp][columns], added in order
        float* const s_part = reinterpret_cast<float*>(s_ring);
        const int columns = (kWarp ? 1 : team) * 32 * C * V, first = static_cast<int>(rank) * columns;
        const int width = lanes * C * V, teams = kWarp ? 32 / lanes : 1;  // (several rows a warp: a team's columns)
        float* const d = s_part + group * 2 * columns + (lane / lanes) * width - first;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int j = my.col(c, i), k = j + my.apart();
                const float2 a = split(dw[c][i]), b = split(dwp[c][i]);
                d[j] = a.x;
                d[k] = a.y;
                d[columns + j] = b.x;
                d[columns + k] = b.y;
            }
        __syncthreads();
        float* const out = p.part + int64_t(block) * 2 * p.N;
        for (int j = threadIdx.x; j < columns && first + j < N; j += blockDim.x) {
            if (kWarp && j >= width) break;
            float a = 0.0f, b = 0.0f;
            for (int g = 0; g < groups; ++g)
                for (int k = 0; k < teams; ++k) {
                    a += s_part[g * 2 * columns + k * width + j];
                    b += s_part[g * 2 * columns + columns + k * width + j];
                }
            out[first + j] = a;
            out[p.N + first + j] = b;
        }
        if constexpr (ALPHA) {
            float a = team_sum<false>(fold(dalpha2), 32);
            if (lane == 0) s_alpha[warp] = a;
            if constexpr (MODE == BN_CLUSTER) cluster_sync_all();
            else __syncthreads();
            if (threadIdx.x == 0 && rank == 0) {
                a = 0.0f;
                for (uint32_t r = 0; r < ctas; ++r)
                    for (int k = 0; k < nw; ++k)
                        a += MODE == BN_CLUSTER ? ld_cluster_f32(mapa_shared(smem_u32(&s_alpha[k]), r)) : s_alpha[k];
                p.part[int64_t(p.parts) * 2 * p.N + block] = a;
            }
        }
    }
    if constexpr (MODE == BN_CLUSTER) cluster_sync_all();  // the sums that another CTA reads stay until it has
}

template <typename T, int C, BnMode MODE, bool ALPHA, bool SHIFT>
cudaError_t launch_bn_bwd_as(BnBwd<T> p, int team, unsigned block, int ctas, int most, int* parts, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const auto kern = bn_bwd_kernel<T, C, MODE, ALPHA, SHIFT>;
    const int warps = block / 32;
    const size_t ring = size_t(bn_bwd_stages(ALPHA)) * (ALPHA ? 5 : 4) * warps * bn_slots(C, SHIFT, MODE == BN_NARROW && C == 1) * 16;
    const size_t sums = size_t(warps) * 2 * 32 * C * V * sizeof(float);
    const size_t smem = std::max(ring, sums);
    if constexpr (MODE == BN_CLUSTER) {
        static DeviceTable<17 * 9> table;  // clusters that run at a time, by warps and CTAs of one
        int device = 0, n = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(ctas * sm_count());
        cfg.blockDim = dim3(block);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = table.get(device, warps * 9 + ctas, &n, [&](int* clusters) {
            cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing);
            if (err == cudaSuccess) err = cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
            return err;
        });
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorNotSupported;
        const int64_t grid = std::min<int64_t>(std::min<int64_t>(p.M, n), most);
        p.parts = *parts = static_cast<int>(grid);
        cfg.gridDim = dim3(static_cast<unsigned>(grid * ctas));
        cfg.stream = stream;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kern, p, team);
    } else {
        static DeviceTable<17> table;
        int n = 0;
        const cudaError_t e = resident_ctas(table, kern, block, smem, kMaxRing, &n);
        if (e != cudaSuccess) return e;
        const int64_t rows = MODE == BN_WIDE ? warps / team : warps * (C > 1 ? 1 : 32 / team);
        const int64_t grid = std::min<int64_t>(std::min<int64_t>((p.M + rows - 1) / rows, int64_t(n) * sm_count()), most);
        p.parts = *parts = static_cast<int>(grid);
        return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, p, team);
    }
}

}  // namespace

// The one-pass kernels, where the row fits one; cudaErrorNotSupported where it does not.
template <typename T, bool SHIFT>
cudaError_t launch_bn_fwd(const BnFwd<T>& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), kMost = 32 / V;
    const int64_t pieces = (p.N + V - 1) / V;
    const int team = team_of(pieces);
    switch ((pieces + team - 1) / team) {
        case 1: return launch_bn_fwd_as<T, 1, false, SHIFT>(p, team, 128, stream);
        case 2: return launch_bn_fwd_as<T, 2, false, SHIFT>(p, team, 128, stream);
        case 3: return launch_bn_fwd_as<T, 3, false, SHIFT>(p, team, 128, stream);
        case 4: return launch_bn_fwd_as<T, 4, false, SHIFT>(p, team, 128, stream);
        case 5: return launch_bn_fwd_as<T, 5, false, SHIFT>(p, team, 128, stream);
        case 6: return launch_bn_fwd_as<T, 6, false, SHIFT>(p, team, 128, stream);
        case 7: return launch_bn_fwd_as<T, 7, false, SHIFT>(p, team, 128, stream);
        case 8: return launch_bn_fwd_as<T, 8, false, SHIFT>(p, team, 128, stream);
        default: break;
    }
    const unsigned block = threads_of(pieces, kMost);
    // three rows of 16 384 two-byte columns, or 8192 of four bytes, fit shared memory; of wider ones of four bytes one
    if (block <= (V == 8 ? 512 : 256)) return launch_bn_fwd_as<T, kMost, true, SHIFT>(p, 32, block, stream);
    if constexpr (V == 4)
        if (block <= 512) return launch_bn_fwd_as<T, kMost, true, SHIFT, 1>(p, 32, block, stream);
    return cudaErrorNotSupported;
}

// At most `most` partial rows; *parts of them are written.
template <typename T, bool ALPHA, bool SHIFT>
cudaError_t launch_bn_bwd(const BnBwd<T>& p, int most, int* parts, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), kC = 2;  // pieces a lane
    const int64_t pieces = (p.N + V - 1) / V;
    if (pieces <= 32) return launch_bn_bwd_as<T, 1, BN_NARROW, ALPHA, SHIFT>(p, team_of(pieces), 256, 1, most, parts, stream);
    if (pieces <= 32 * kC) return launch_bn_bwd_as<T, kC, BN_NARROW, ALPHA, SHIFT>(p, 32, 512, 1, most, parts, stream);
    const int64_t team = (pieces + 32 * kC - 1) / (32 * kC);  // warps of a row
    // Two-byte types: a warp a row up to 24 columns a lane (65536 x 768: 93 us, 111 in two warps of 16), and 32
    // columns a lane where 16 would leave a seventh of the lanes idle (131072 x 1600: 400 us, 433) or make a whole
    // CTA one group (8192 x 8192: 129, 142); where they fill the lanes 16 are better (65536 x 2048: 239, 252), and
    // off the grid (65536 x 1601: 401, 457 before last granules were copied in part).
    if constexpr (V == 8) {
        if (pieces <= 96) return launch_bn_bwd_as<T, 3, BN_NARROW, ALPHA, SHIFT>(p, 32, 256, 1, most, parts, stream);
        if constexpr (!SHIFT) {
            const int64_t four = (pieces + 127) / 128;
            if (four <= 8 && four * 2 <= team && (pieces * 20 < team * 64 * 17 || team > 8)) {
                const unsigned block = static_cast<unsigned>(8 / four * four) * 32;
                return launch_bn_bwd_as<T, 4, BN_WIDE, ALPHA, SHIFT>(p, static_cast<int>(four), block, 1, most, parts, stream);
            }
        }
    }
    if (team <= 16) {
        const unsigned block = static_cast<unsigned>(16 / team * team) * 32;
        return launch_bn_bwd_as<T, kC, BN_WIDE, ALPHA, SHIFT>(p, static_cast<int>(team), block, 1, most, parts, stream);
    }
    for (int ctas = 2; ctas <= 8; ctas *= 2)  // (portable cluster sizes)
        if (team <= 16 * ctas) {
            const unsigned block = static_cast<unsigned>((team + ctas - 1) / ctas) * 32;
            return launch_bn_bwd_as<T, kC, BN_CLUSTER, ALPHA, SHIFT>(p, 32, block, ctas, most, parts, stream);
        }
    return cudaErrorNotSupported;
}

}  // namespace fp8q
