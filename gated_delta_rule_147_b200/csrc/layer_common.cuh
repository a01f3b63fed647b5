// Shared device helpers of the layer operators (short convolution, selective
// scan, query/key norm): vector loads and stores with conversion, the
// activations, packed fp32 pairs, and the launch as a programmatic dependent.
#pragma once

#include <initializer_list>

#include "common.cuh"

namespace gdr {

// V consecutive elements as floats; one or two 16-byte (or one 8-byte) loads
// when V > 1, which needs the address aligned to the access.
template <typename T, int V> struct VecIO;
template <typename T> struct VecIO<T, 1> {
    static __device__ __forceinline__ void load(float* f, const T* p) { f[0] = to_f32(*p); }
    static __device__ __forceinline__ void store(T* p, const float* f) { *p = from_f32<T>(f[0]); }
};
template <> struct VecIO<float, 2> {
    static __device__ __forceinline__ void load(float* f, const float* p) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[0] = v.x; f[1] = v.y;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    }
};
template <> struct VecIO<float, 4> {
    static __device__ __forceinline__ void load(float* f, const float* p) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct VecIO<float, 8> {
    static __device__ __forceinline__ void load(float* f, const float* p) {
        VecIO<float, 4>::load(f, p);
        VecIO<float, 4>::load(f + 4, p + 4);
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        VecIO<float, 4>::store(p, f);
        VecIO<float, 4>::store(p + 4, f + 4);
    }
};
__device__ __forceinline__ void unpack_bf16x2(uint32_t u, float& lo, float& hi) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}
template <> struct VecIO<__nv_bfloat16, 2> {
    static __device__ __forceinline__ void load(float* f, const __nv_bfloat16* p) {
        unpack_bf16x2(*reinterpret_cast<const uint32_t*>(p), f[0], f[1]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
    }
};
template <> struct VecIO<__nv_bfloat16, 4> {
    static __device__ __forceinline__ void load(float* f, const __nv_bfloat16* p) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        unpack_bf16x2(u.x, f[0], f[1]);
        unpack_bf16x2(u.y, f[2], f[3]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
};
template <> struct VecIO<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(float* f, const __nv_bfloat16* p) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        unpack_bf16x2(u.x, f[0], f[1]);
        unpack_bf16x2(u.y, f[2], f[3]);
        unpack_bf16x2(u.z, f[4], f[5]);
        unpack_bf16x2(u.w, f[6], f[7]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// V consecutive elements as loaded, so that rows requested ahead of their use
// cost no more registers than their bytes.
template <typename T, int V> struct RawVec {
    static constexpr int kWords = V * sizeof(T) >= 4 ? V * sizeof(T) / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V * sizeof(T) == 2) {
            w[0] = *reinterpret_cast<const unsigned short*>(p);
        } else if constexpr (kWords == 1) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void set(int i, T x) {  // into zeros
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x);
        else w[i / 2] |= (uint32_t)__bfloat16_as_ushort(x) << (i % 2 * 16);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-x) from the hardware exponential and reciprocal; e^-x = inf
// gives 0. Relative error a few 2^-24, and for negative x about 1.3 |x| 2^-24 more:
// the product x log2(e) and log2(e) itself are rounded.
__device__ __forceinline__ float sigmoidf_fast(float x) {
    return rcp_approx(1.f + ex2_approx(-x * kLog2e));
}

// The smaller and the larger one; NaN where either is (fminf and fmaxf drop it).
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// ---- packed pairs of fp32 (one instruction for two multiply-adds) ----
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 ex2_pair(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2_approx(a), ex2_approx(b));
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}
__device__ __forceinline__ f2 both2(float a) { return pack2(a, a); }
__device__ __forceinline__ f2 sigmoid2(f2 x) {  // sigmoidf_fast of each
    const f2 q = add2(ex2_pair(mul2(x, both2(-kLog2e))), both2(1.f));
    float a, b;
    unpack2(q, a, b);
    return pack2(rcp_approx(a), rcp_approx(b));
}

// Decay e^(dt A), given A log2(e). The hardware exponential's results lie on
// average 0.3 2^-24 below the true ones (measured over arguments of -1 to 0, root
// mean square 0.6); that is small, but a slow state is multiplied by its decay
// thousands of times, and the state came out twice as far off as with correctly
// rounded exponentials. So the argument gets the 0.32 2^-24 / ln 2 back, in the
// multiply-add that forms it; an argument of 0 still gives 1.
__device__ __forceinline__ float decay_rate(float A) {  // A log2(e)
    // A = -inf (a state that holds one token) times dt = 0 of a padded token would be
    // NaN; the lowest number gives the same decays
    return max_nan(A * kLog2e, -3.402823466e38f);
}
__device__ __forceinline__ f2 decay2(f2 dt, f2 a) { return ex2_pair(fma2(dt, a, both2(2.75e-8f))); }

// log(1 + e^x) = max(x, 0) + log1p(y), y = e^-|x| in (0, 1], with log1p(y) = y Q(y):
// relative accuracy is kept for y -> 0 (large negative x), which log(1 + y)
// loses. Q is the polynomial of degree 8 with the least greatest relative error
// on [0, 1] (Remez exchange on log1p(y) / y): 3.1e-8, with fp32 arithmetic below
// 3 2^-24. An error in a step size goes into every later state, so y gets back
// what the product x log2(e) and log2(e) itself lost in rounding, and most of the
// exponential's mean error (0.8 2^-24 below over arguments from -8 to -1). |x| is
// held to 128, where y is 0 already: the product and its rest must stay finite, for
// a step input of -inf or the type's lowest number masks its token.
// `sig`: the derivative, 1 / (1 + y) or y / (1 + y).
__device__ __forceinline__ f2 exp_neg2(f2 x) {  // e^-x, 0 <= x <= 128
    const f2 t = mul2(x, both2(kLog2e));  // 2^-t, and 2^r with the rest r of the exponent
    f2 r = fma2(x, both2(-kLog2e), t);
    r = fma2(x, both2(-1.925963033500e-08f), add2(r, both2(5e-8f)));
    float a, b;
    unpack2(t, a, b);
    const f2 y = pack2(ex2_approx(-a), ex2_approx(-b));
    return fma2(mul2(y, both2(0.69314718f)), r, y);
}
struct StepCurve { f2 dt, sig; };
template <bool SIG> __device__ __forceinline__ StepCurve softplus2(f2 x) {
    float a, b;
    unpack2(x, a, b);
    const f2 y = exp_neg2(pack2(min_nan(fabsf(a), 128.f), min_nan(fabsf(b), 128.f)));
    float ya, yb;
    unpack2(y, ya, yb);
    f2 r = both2(0.0052326940931379795f);
    r = fma2(r, y, both2(-0.029505237936973572f));
    r = fma2(r, y, both2(0.07822594791650772f));
    r = fma2(r, y, both2(-0.13663245737552643f));
    r = fma2(r, y, both2(0.19106006622314453f));
    r = fma2(r, y, both2(-0.2484298199415207f));
    r = fma2(r, y, both2(0.3331909775733948f));
    r = fma2(r, y, both2(-0.4999949336051941f));
    r = fma2(r, y, both2(0.9999999403953552f));
    StepCurve c;
    c.dt = fma2(r, y, pack2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
    c.sig = both2(1.f);
    if (SIG) c.sig = mul2(pack2(rcp_approx(1.f + ya), rcp_approx(1.f + yb)), pack2(a < 0.f ? ya : 1.f, b < 0.f ? yb : 1.f));
    return c;
}
// One value (the pair form takes registers that the single-token kernel needs
// for its loads in flight: 34.6 against 29.5 us).
__device__ __forceinline__ float softplusf(float x) {
    const float y = expf(-fabsf(x));
    float r = 0.0052326940931379795f;
    r = fmaf(r, y, -0.029505237936973572f);
    r = fmaf(r, y, 0.07822594791650772f);
    r = fmaf(r, y, -0.13663245737552643f);
    r = fmaf(r, y, 0.19106006622314453f);
    r = fmaf(r, y, -0.2484298199415207f);
    r = fmaf(r, y, 0.3331909775733948f);
    r = fmaf(r, y, -0.4999949336051941f);
    r = fmaf(r, y, 0.9999999403953552f);
    return fmaf(r, y, fmaxf(x, 0.f));
}

// V channels (even) of one row, as loaded: a vector (kWholeRow), pairs, or one
// element at a time where only that is aligned; of the last two `left` elements
// exist, the others are 0.
enum { kSingleRow = 0, kWholeRow = 1, kPairRow = 2 };
template <typename T, int V, int HOW> struct RowIO {
    RawVec<T, V> v;
    __device__ __forceinline__ void zero() { v.zero(); }
    __device__ __forceinline__ void load(const T* p, int left) {
        if constexpr (HOW == kWholeRow) {
            v.load(p);
        } else if constexpr (HOW == kPairRow) {
            constexpr int kWords = RawVec<T, 2>::kWords;
            v.zero();
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if (2 * i >= left) continue;
                RawVec<T, 2> r;
                r.load(p + 2 * i);
#pragma unroll
                for (int j = 0; j < kWords; ++j) v.w[i * kWords + j] = r.w[j];
            }
        } else {
            v.zero();
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < left) v.set(i, p[i]);
        }
    }
    __device__ __forceinline__ f2 pair(int i) const { return pack2(v.get(2 * i), v.get(2 * i + 1)); }
    static __device__ __forceinline__ void store(T* p, const f2 (&f)[V / 2], int left) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) unpack2(f[i], s[2 * i], s[2 * i + 1]);
        if constexpr (HOW == kWholeRow) {
            VecIO<T, V>::store(p, s);
        } else if constexpr (HOW == kPairRow) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                if (2 * i < left) VecIO<T, 2>::store(p + 2 * i, s + 2 * i);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < left) p[i] = from_f32<T>(s[i]);
        }
    }
};

// Tokens of sequence b: lengths[b] held to [0, T], or T without lengths.
__device__ __forceinline__ int seq_len(const int* lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// A kernel launched with launch_dependent() starts while the previous kernel
// of the stream drains; nothing may be read before this returns.
__device__ __forceinline__ void dependent_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependent_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Host checks shared by the entry points.
// Tokens, channels and sequences are counted in int, and some loops and roundings
// count a little past the last one (a chunk, a step on its way).
constexpr int kMaxAxis = 0x7fffffff - 4096;
inline bool axes_fit(std::initializer_list<long long> axes) {
    for (long long n : axes)
        if (n > kMaxAxis) return false;
    return true;
}
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t dtype_size(int dtype) { return dtype == GDR_BF16 ? 2 : 4; }
inline bool dtype_ok(int dtype) { return dtype == GDR_BF16 || dtype == GDR_FP32; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace gdr
