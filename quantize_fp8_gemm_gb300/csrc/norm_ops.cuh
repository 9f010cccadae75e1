// norm_ops.cuh -- element types, the counter-based generator and the quantize
// epilogue shared by the layer norm (norm_fwd.cu, norm_bwd.cu) and dropout
// (dropout.cu) kernels.
#pragma once

#include "common.cuh"
#include "quant_ops.cuh"

#include <type_traits>

namespace fp8q {

// ------------------------------------------------------------ element types --
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Round to nearest even; a half-precision overflow gives infinity.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The float32 value of v rounded to T.
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f32(from_f32<T>(v)); }

// A parameter vector of either type: float32, or the activations' type T.
template <typename T>
struct Params {
    const void* p;  // NULL: every value is `none`
    bool f32;
    float none;
    __device__ __forceinline__ float at(int64_t j) const {
        if (p == nullptr) return none;
        return f32 ? static_cast<const float*>(p)[j] : to_f32(static_cast<const T*>(p)[j]);
    }
};

// V adjacent elements of a row: 16 bytes in one access, or one element.
template <typename T, int V>
struct Piece {
    static_assert(V * sizeof(T) == 16, "16-byte pieces or single elements");
    uint4 raw;
    __device__ __forceinline__ void load(const T* p) { raw = ld_stream_v4(p); }
    __device__ __forceinline__ void store(T* p) const { st_v4(p, raw); }
    __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void unpack(float (&v)[V]) const {
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(u[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                v[2 * i] = bf16lo_to_f32(u[i]);
                v[2 * i + 1] = bf16hi_to_f32(u[i]);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&v)[V]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                u[i] = __float_as_uint(v[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                u[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        raw = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <typename T>
struct Piece<T, 1> {
    T raw;
    __device__ __forceinline__ void load(const T* p) { raw = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = raw; }
    __device__ __forceinline__ void zero() { raw = from_f32<T>(0.0f); }
    __device__ __forceinline__ void unpack(float (&v)[1]) const { v[0] = to_f32(raw); }
    __device__ __forceinline__ void pack(const float (&v)[1]) { raw = from_f32<T>(v[0]); }
};

// Two float32 values in one 64-bit register pair; each lane of an operation is
// the IEEE operation rounded once, at half the instructions.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair_of(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// A 16-byte piece as pairs, and back.
template <typename T, int V>
__device__ __forceinline__ void unpack2(const Piece<T, V>& q, f32x2 (&v)[V / 2]) {
    float f[V];
    q.unpack(f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = pair_of(f[2 * i], f[2 * i + 1]);
}
template <typename T, int V>
__device__ __forceinline__ void pack2(Piece<T, V>& q, const f32x2 (&v)[V / 2]) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 a = split(v[i]);
        f[2 * i] = a.x;
        f[2 * i + 1] = a.y;
    }
    q.pack(f);
}

// V parameters from column j (16-byte accesses need the vector 16-byte aligned).
template <typename T, int V>
__device__ __forceinline__ void load_params(const Params<T>& w, int64_t j, float (&v)[V]) {
    if (w.p == nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = w.none;
    } else if constexpr (V == 1) {
        v[0] = w.at(j);
    } else if (w.f32) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + j + i));
            v[i] = f.x;
            v[i + 1] = f.y;
            v[i + 2] = f.z;
            v[i + 3] = f.w;
        }
    } else {
        Piece<T, V> q;
        q.raw = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w.p) + j));
        q.unpack(v);
    }
}

// ----------------------------------------------------------------- dropout --
// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit
// products over a 128-bit counter under a 64-bit key that grows by a constant
// each round.  The key is the seed; the counter is (column / 4, row, offset
// low, offset high), so a block gives the four words of columns 4j .. 4j + 3
// of one row, and the mask depends on seed, offset, row and column alone:
// not on the element type, the strides, the launch shape or the kernel.
struct Philox {
    uint32_t k0, k1, o0, o1;
    Philox() = default;
    __device__ __forceinline__ explicit Philox(const uint64_t* rng) {
        const uint64_t seed = rng[0], off = rng[1];
        k0 = static_cast<uint32_t>(seed);
        k1 = static_cast<uint32_t>(seed >> 32);
        o0 = static_cast<uint32_t>(off);
        o1 = static_cast<uint32_t>(off >> 32);
    }
    __device__ __forceinline__ uint4 block(uint32_t quad, uint32_t row) const {
        uint32_t c0 = quad, c1 = row, c2 = o0, c3 = o1, a = k0, b = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
            const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
            c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a;
            c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ b;
            c1 = static_cast<uint32_t>(p1);
            c3 = static_cast<uint32_t>(p0);
            a += 0x9E3779B9u;
            b += 0xBB67AE85u;
        }
        return make_uint4(c0, c1, c2, c3);
    }
};

// Drop probability as the kernels use it.  An element is dropped when its word
// is <= last (= round(p 2^32) - 1), i.e. below round(p 2^32); p that rounds to
// no word at all runs without a generator (on = false).
struct Dropout {
    const uint64_t* rng;
    uint32_t last;
    float inv;  // float32(1 / (1 - p)); 0 for p = 1, where every element is dropped
    bool on;
};

// Host: false if p is not in [0, 1].
inline bool make_dropout(double p, const void* rng, Dropout* d) {
    if (!(p >= 0.0 && p <= 1.0)) return false;
    const double words = p * 4294967296.0;
    uint64_t n = static_cast<uint64_t>(words);  // round half to even, as the documented formula rounds
    const double rest = words - static_cast<double>(n);
    if (rest > 0.5 || (rest == 0.5 && (n & 1u))) ++n;
    d->rng = static_cast<const uint64_t*>(rng);
    d->on = n > 0;
    d->last = n > 0 ? static_cast<uint32_t>(n - 1) : 0u;
    d->inv = p < 1.0 ? static_cast<float>(1.0 / (1.0 - p)) : 0.0f;
    return true;
}

__device__ __forceinline__ uint32_t word_of(uint4 w, int i) {
    return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// keep ? x * inv : 0.  A dropped element is 0 whatever x holds.
__device__ __forceinline__ float dropped(float x, uint32_t word, const Dropout& d) {
    return word > d.last ? __fmul_rn(x, d.inv) : 0.0f;
}

// The generator words of the V columns from j of a row (V = 1: the word of column j).
template <int V>
__device__ __forceinline__ void words_at(const Philox& g, uint32_t j, uint32_t row, uint32_t (&w)[V]) {
    if constexpr (V == 1) {
        w[0] = word_of(g.block(j >> 2, row), j & 3);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const uint4 b = g.block((j + i) >> 2, row);
            w[i] = b.x;
            w[i + 1] = b.y;
            w[i + 2] = b.z;
            w[i + 3] = b.w;
        }
    }
}

// -------------------------------------------------------- quantize epilogue --
// The framework's cast of the rounded output: v = y * s, q = FP8(v), max |y|
// (as float32 bits: those of non-negative floats order like the values, and a
// NaN orders above infinity, as in the quantize kernels), #{|v| > max}.
struct QuantOut {
    const float* scale;
    uint8_t* q;
    float* amax;
    unsigned long long* sat;
    int fmt;
    bool on;
};

__device__ __forceinline__ uint16_t cast_pair(float v0, float v1, int fmt) {
    return fmt == FP8Q_E5M2 ? cvt_fp8x2<FP8Q_E5M2>(v0, v1) : cvt_fp8x2<FP8Q_E4M3>(v0, v1);
}

// Scale and cast V values of the rounded output from a row's column j; folds
// their magnitudes and saturations into amax / nsat.
template <typename T, int V>
__device__ __forceinline__ void quant_piece(const QuantOut& o, float s, const Piece<T, V>& y, uint8_t* dst,
                                            uint32_t& amax, uint32_t& nsat) {
    float f[V], v[V];
    y.unpack(f);
    const float fmax = fp8_max_value(o.fmt);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = __fmul_rn(f[i], s);
        amax = max(amax, __float_as_uint(fabsf(f[i])));
        nsat += fabsf(v[i]) > fmax;
    }
    if (dst == nullptr) return;
    if constexpr (V == 1) {
        *dst = static_cast<uint8_t>(cast_pair(v[0], 0.0f, o.fmt));
    } else {
        uint32_t q[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            q[i] = cast_pair(v[4 * i], v[4 * i + 1], o.fmt) |
                   (static_cast<uint32_t>(cast_pair(v[4 * i + 2], v[4 * i + 3], o.fmt)) << 16);
        if constexpr (V == 8) st_v2(dst, make_uint2(q[0], q[1]));
        else *reinterpret_cast<uint32_t*>(dst) = q[0];
    }
}

// The same for the 8 packed BF16 values of a piece, magnitudes folded into two
// 16-bit lanes.  Saturations are counted only where the largest magnitude can
// saturate (a NaN among them takes the counting route too).
template <int FMT>
__device__ __forceinline__ void quant_bf16x8(float s, uint4 y, uint8_t* dst, uint32_t& amax2, uint32_t& nsat) {
    uint32_t m2 = __vmaxu2(__vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu),
                           __vmaxu2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu));
    amax2 = __vmaxu2(amax2, m2);
    if (!(__fmul_rn(__uint_as_float(max16x2(m2) << 16), s) <= fp8_max_value(FMT))) nsat += sat_count8<FMT>(y, s);
    if (dst != nullptr) st_v2(dst, cast8_codes<FMT>(y, s));
}

// A warp's maximum and count into the call's accumulators.  The maximum only
// grows, so a warp whose own is no larger than a value read earlier has
// nothing to add: of tens of thousands of warps a few reach the atomic.
__device__ __forceinline__ void publish_quant(const QuantOut& o, uint32_t amax, uint32_t nsat) {
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    nsat = __reduce_add_sync(0xFFFFFFFFu, nsat);
    if ((threadIdx.x & 31) != 0) return;
    unsigned* a = reinterpret_cast<unsigned*>(o.amax);
    if (a && amax > *reinterpret_cast<volatile unsigned*>(a)) atomicMax(a, amax);
    if (o.sat && nsat) atomicAdd(o.sat, static_cast<unsigned long long>(nsat));
}

// Zeroes the accumulators of a call that does not accumulate.  One launch for
// both words, and one the next kernel's launch overlaps.
__global__ void clear_quant_kernel(float* amax, unsigned long long* sat);

inline bool is_dtype(int t) { return t == FP8Q_BF16 || t == FP8Q_FP16 || t == FP8Q_FP32; }
inline size_t dtype_size(int t) { return t == FP8Q_FP32 ? 4 : 2; }
// Whether a tensor's rows (NULL: no tensor) all start on 16-byte boundaries.
inline bool rows16(const void* p, int64_t ld, size_t es) {
    return p == nullptr || (aligned16(p) && (static_cast<uint64_t>(ld) * es) % 16 == 0);
}
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Sum over the CTA's threads of two values, in every thread; the order of the
// additions depends on blockDim.x alone.  `s` holds 2 * 32 + 2 floats.
__device__ __forceinline__ float2 block_sum2(float a, float b, float* s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    __syncthreads();  // the previous sum's readers are done with s
    if (lane == 0) { s[warp] = a; s[32 + warp] = b; }
    __syncthreads();
    a = lane < nw ? s[lane] : 0.0f;
    b = lane < nw ? s[32 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    return make_float2(a, b);
}

}  // namespace fp8q
