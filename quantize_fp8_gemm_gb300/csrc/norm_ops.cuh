// norm_ops.cuh -- element types, the counter-based generator and the quantize
// epilogue shared by the layer norm (norm_fwd.cu, norm_bwd.cu) and dropout
// (dropout.cu) kernels.
#pragma once

#include "common.cuh"
#include "launch_table.cuh"
#include "quant_ops.cuh"

#include <algorithm>
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
    bool aligned;   // on a 16-byte boundary
    __device__ __forceinline__ float at(int64_t j) const {
        if (p == nullptr) return none;
        return f32 ? static_cast<const float*>(p)[j] : to_f32(static_cast<const T*>(p)[j]);
    }
};

// V adjacent elements of a row, 16 bytes.
template <typename T, int V>
struct Piece {
    static_assert(V * sizeof(T) == 16, "16-byte pieces");
    uint4 raw;
    __device__ __forceinline__ void load(const T* p) { raw = ld_once_v4(p); }  // an output may replace an input
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

// V parameters from column j.  ANY: the vector may sit anywhere and end inside
// the piece (n columns; those past it are 0), and goes element by element then.
template <typename T, int V, bool ANY>
__device__ __forceinline__ void load_params2(const Params<T>& w, int j, int n, f32x2 (&v)[V / 2]) {
    float f[V];
    if (w.p == nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = w.none;
    } else if (ANY && (!w.aligned || j + V > n)) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = j + i < n ? w.at(j + i) : 0.0f;
    } else if (w.f32) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + j + i));
            f[i] = q.x;
            f[i + 1] = q.y;
            f[i + 2] = q.z;
            f[i + 3] = q.w;
        }
    } else {
        Piece<T, V> q;
        q.raw = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w.p) + j));
        q.unpack(f);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = pair_of(f[2 * i], f[2 * i + 1]);
}

// ------------------------------------------- rows off the 16-byte grid (SHIFT) --
// A row that does not start on a 16-byte boundary is moved in the granules (16
// aligned bytes) that it touches, and its pieces of V columns are cut from two
// neighbouring ones, so the arithmetic and its order do not depend on where the
// rows lie.  A granule that holds an element of the row is read whole; its other
// bytes are not used.  Writes touch the row's own elements only.

// Bytes mis .. mis + 15 of a:b (0 <= mis < 16; whole elements of ES = 2 or 4 bytes).
template <int ES>
__device__ __forceinline__ uint4 cut16(uint4 a, uint4 b, uint32_t mis) {
    uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (mis & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) u[i] = u[i + 2];
    }
    if (mis & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
    }
    if constexpr (ES == 4) return make_uint4(u[0], u[1], u[2], u[3]);
    const uint32_t bits = (mis & 3) * 8;
    return make_uint4(__funnelshift_r(u[0], u[1], bits), __funnelshift_r(u[1], u[2], bits),
                      __funnelshift_r(u[2], u[3], bits), __funnelshift_r(u[3], u[4], bits));
}

// Bytes between a row's granule boundary and its first element.
template <typename T>
__device__ __forceinline__ uint32_t granule_offset(const T* start) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(start) & 15);
}
// cp.async, to shared address `slot`, of granule k of a row whose first granule is
// at `first`, and of granule k + 1 into the next slot if `two`.  INSIDE: both hold
// elements of the row; otherwise one that begins at or after `end` bytes from
// `first` is zeros (no byte of it is read).
template <bool INSIDE>
__device__ __forceinline__ void copy_granules(uint32_t slot, const uint8_t* first, int k, int end, bool two) {
    const uint8_t* at = first + static_cast<int64_t>(k) * 16;
    if constexpr (INSIDE) {
        cp_async16(slot, at);
        if (two) cp_async16(slot + 16, at + 16);
    } else {
        const bool has = k * 16 < end, has2 = k * 16 + 16 < end;
        cp_async16_or_zero(slot, has ? at : first, has);
        if (two) cp_async16_or_zero(slot + 16, has2 ? at + 16 : first, has2);
    }
}
// This lane's piece from the ring: its slot, or cut from its slot and the next.
template <typename T, bool SHIFT>
__device__ __forceinline__ uint4 read_piece(const uint4* slot, uint32_t mis) {
    if constexpr (SHIFT) return cut16<sizeof(T)>(slot[0], slot[1], mis);
    return slot[0];
}
// Zero the columns from `valid` on.
template <int V>
__device__ __forceinline__ void zero_from(f32x2 (&v)[V / 2], int valid) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 f = split(v[i]);
        v[i] = pair_of(2 * i < valid ? f.x : 0.0f, 2 * i + 1 < valid ? f.y : 0.0f);
    }
}

// The same of a packed piece.
template <typename T, int V>
__device__ __forceinline__ void clear_from(Piece<T, V>& q, int valid) {
    float f[V];
    q.unpack(f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i < valid ? f[i] : 0.0f;
    q.pack(f);
}

// Elements lo .. hi - 1 of a piece, one by one, to dst + their index.
template <typename T>
__device__ __forceinline__ void store_elements(T* dst, uint4 q, int lo, int hi) {
    constexpr int V = 16 / sizeof(T);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i < lo || i >= hi) continue;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint32_t*>(dst + i) = u[i];
        else
            *reinterpret_cast<uint16_t*>(dst + i) = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
    }
}

// Store a warp's pieces: this lane's is piece k of the row at `start`, with
// `valid` elements (0: none; fewer than V only in the row's last piece).  Lanes
// hold adjacent pieces, and a call for the warp's next 32 pieces follows with the
// same `carry`.  All lanes of the warp call it.  A lane writes the granule in
// which its piece begins, whose first bytes are the end of the piece before (of
// lane 0's from the call before); where a warp's part of the row begins (`head`),
// and what is left of the last piece of it (`tail`), go element by element.
// HEAD, TAIL: whether the call's pieces can be such.
template <typename T, bool HEAD, bool TAIL>
__device__ __forceinline__ void store_shifted(uint4 q, uint4& carry, T* start, int k, int valid, bool head, bool tail) {
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 31, from = (lane + 31) & 31;
    uint4 prev;
    prev.x = __shfl_sync(0xFFFFFFFFu, q.x, from);
    prev.y = __shfl_sync(0xFFFFFFFFu, q.y, from);
    prev.z = __shfl_sync(0xFFFFFFFFu, q.z, from);
    prev.w = __shfl_sync(0xFFFFFFFFu, q.w, from);
    const uint4 next_carry = prev;
    if (lane == 0) prev = carry;
    carry = next_carry;
    if (valid <= 0) return;
    T* dst = start + static_cast<int64_t>(k) * V;
    const uint32_t mis = granule_offset(start);
    const int lead = (16 - static_cast<int>(mis)) / static_cast<int>(sizeof(T));  // of this piece in its first granule
    const bool whole = (!HEAD || !head || mis == 0) && (!TAIL || valid >= lead);
    if (whole) {
        const uint4 cut = cut16<sizeof(T)>(prev, q, 16 - mis);
        st_v4(reinterpret_cast<uint8_t*>(dst) - mis, mis ? cut : q);
    }
    if constexpr (HEAD || TAIL) {
        // (mis = 0: lead = V, and a piece that ends the row early is its first `valid` elements)
        if (!whole) {
            if (mis != 0 && !(HEAD && head)) store_elements<T>(dst - V, prev, lead, V);
            store_elements<T>(dst, q, 0, valid < lead ? valid : lead);
        }
        if (TAIL && tail) store_elements<T>(dst, q, lead, valid);
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
//
// The 32 x 32 -> 64 bit products bound these kernels next to the memory (each
// takes the multiply pipe four cycles a warp), so those that do not depend on
// the block are formed once: round 1's second product (of the offset) per
// thread, round 2's first one (of the row) per row.  Round 1's first product,
// of the column quad, is linear in it: a caller adds kPhiloxM0 times a step
// instead.  That leaves 17 of 20 products a block.
constexpr uint64_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;

struct Philox {
    uint32_t k0, k1, o1;
    uint64_t off;           // M1 * (offset low half)
    uint32_t a[9], b[9];    // the keys of rounds 2 .. 10
    Philox() = default;
    __device__ __forceinline__ explicit Philox(const uint64_t* rng) {
        const uint64_t seed = rng[0], o = rng[1];
        k0 = static_cast<uint32_t>(seed);
        k1 = static_cast<uint32_t>(seed >> 32);
        o1 = static_cast<uint32_t>(o >> 32);
        off = kPhiloxM1 * static_cast<uint32_t>(o);
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            a[i] = k0 + (i + 1) * 0x9E3779B9u;
            b[i] = k1 + (i + 1) * 0xBB67AE85u;
        }
    }
    // Round 2's product of the row: a row's blocks share it.
    __device__ __forceinline__ uint64_t row(uint32_t i) const {
        return kPhiloxM0 * (static_cast<uint32_t>(off >> 32) ^ i ^ k0);
    }
    // The block of a column quad; quad_m0 = M0 * quad.
    __device__ __forceinline__ uint4 block(uint64_t quad_m0, uint64_t row_m0) const {
        const uint64_t p = kPhiloxM1 * (static_cast<uint32_t>(quad_m0 >> 32) ^ o1 ^ k1);
        uint32_t c0 = static_cast<uint32_t>(p >> 32) ^ static_cast<uint32_t>(off) ^ a[0], c1 = static_cast<uint32_t>(p);
        uint32_t c2 = static_cast<uint32_t>(row_m0 >> 32) ^ static_cast<uint32_t>(quad_m0) ^ b[0],
                 c3 = static_cast<uint32_t>(row_m0);
#pragma unroll
        for (int i = 1; i < 9; ++i) {
            const uint64_t p0 = kPhiloxM0 * c0, p1 = kPhiloxM1 * c2;
            c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a[i];
            c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ b[i];
            c1 = static_cast<uint32_t>(p1);
            c3 = static_cast<uint32_t>(p0);
        }
        return make_uint4(c0, c1, c2, c3);
    }
    __device__ __forceinline__ uint4 at(uint32_t quad, uint32_t i) const { return block(kPhiloxM0 * quad, row(i)); }
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

// The generator words of V columns whose first quad's M0 * quad is given.
template <int V>
__device__ __forceinline__ void words_at(const Philox& g, uint64_t quad_m0, uint64_t row_m0, uint32_t (&w)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const uint4 b = g.block(quad_m0 + (i / 4) * kPhiloxM0, row_m0);
        w[i] = b.x;
        w[i + 1] = b.y;
        w[i + 2] = b.z;
        w[i + 3] = b.w;
    }
}

// A pair of products x * inv, 0 where dropped.
__device__ __forceinline__ f32x2 dropped2(f32x2 scaled, uint32_t word0, uint32_t word1, const Dropout& d) {
    const float2 f = split(scaled);
    return pair_of(word0 > d.last ? f.x : 0.0f, word1 > d.last ? f.y : 0.0f);
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

// Scale and cast the first `valid` of V values of the rounded output; folds their
// magnitudes and saturations into amax / nsat.  `whole`: dst takes all V codes
// in one store.
template <typename T, int V>
__device__ __forceinline__ void quant_piece(const QuantOut& o, float s, const Piece<T, V>& y, uint8_t* dst, int valid,
                                            bool whole, uint32_t& amax, uint32_t& nsat) {
    float f[V], v[V];
    y.unpack(f);
    const float fmax = fp8_max_value(o.fmt);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = __fmul_rn(f[i], s);
        if (i < valid) {
            amax = max(amax, __float_as_uint(fabsf(f[i])));
            nsat += fabsf(v[i]) > fmax;
        }
    }
    if (dst == nullptr) return;
    uint32_t q[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        q[i] = cast_pair(v[4 * i], v[4 * i + 1], o.fmt) |
               (static_cast<uint32_t>(cast_pair(v[4 * i + 2], v[4 * i + 3], o.fmt)) << 16);
    if (whole) {
        if constexpr (V == 8) st_v2(dst, make_uint2(q[0], q[1]));
        else *reinterpret_cast<uint32_t*>(dst) = q[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) dst[i] = static_cast<uint8_t>(q[i / 4] >> (8 * (i & 3)));
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
// Slots that a warp's ring has of one piece index: with SHIFT one more granule a
// row (33 for one row of 32 pieces, up to 64 where every lane has a row).
__host__ __device__ constexpr int warp_slots(bool shift, bool rows) { return !shift ? 32 : rows ? 64 : 33; }
// Lanes of a warp that take a row of so many pieces: a power of two, 32 at most.
inline int team_of(int64_t pieces) {
    int team = 1;
    while (team < 32 && team < pieces) team *= 2;
    return team;
}
// Threads of a CTA that takes a row at c pieces a thread.
inline unsigned threads_of(int64_t pieces, int c) { return static_cast<unsigned>((pieces + 32 * c - 1) / (32 * c)) * 32; }
constexpr int kMaxRing = 208 * 1024;  // dynamic shared memory that a ring may take
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// *n = CTAs of `kern`, of `block` threads with `smem` bytes, that run at a time on a
// multiprocessor of the current device; on the first call there the kernel is
// allowed `most` bytes.
template <typename Kern>
inline cudaError_t resident_ctas(DeviceTable<17>& table, Kern kern, unsigned block, size_t smem, int most, int* n) {
    int device = 0;
    const cudaError_t got = cudaGetDevice(&device);
    if (got != cudaSuccess) return got;
    return table.get(device, static_cast<int>(block / 32), n, [&](int* ctas) {
        cudaError_t e = most ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) : cudaSuccess;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kern, static_cast<int>(block), smem);
        *ctas = std::max(*ctas, 1);
        return e;
    });
}

// The rows that a thread comes to, `stride` apart.  RUN: the address is carried
// from row to row (two registers more, and no 64-bit product a row: worth it
// where a row is few pieces a lane).
template <typename T, bool RUN>
struct RowWalk {
    T* p;
    int64_t step;
    __device__ __forceinline__ RowWalk(T* base, int64_t ld, uint32_t row0, uint32_t stride)
        : p(RUN ? base + row0 * ld : base), step(RUN ? stride * ld : ld) {}
    __device__ __forceinline__ T* at(uint32_t row) const { return RUN ? p : p + row * step; }
    __device__ __forceinline__ void next() {
        if constexpr (RUN) p += step;
    }
};

// Sum over the lanes of a warp, or (PART) of each team of `team` of them (a power
// of two), in every lane; the order of the additions depends on the team alone.
template <bool PART>
__device__ __forceinline__ float team_sum(float v, int team) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v += !PART || o < team ? other : 0.0f;
    }
    return v;
}

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
