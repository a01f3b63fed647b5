// Per-head norm of queries and keys, with the position rotation in the same
// pass, and its backward.
//
// Per row x of d elements (one token of one head):
//   L2:   n = x / max(|x|, eps)             RMS:  n = w . x / sqrt(mean(x^2) + eps)
//   rotation of the first `rot` elements in pairs (x1, x2) by the angle
//   pos * f_i: (x1 cos - x2 sin, x2 cos + x1 sin), pairs (i, i + rot/2) in the
//   half layout and (2i, 2i + 1) in the interleaved one;
//   q rows are then multiplied by q_scale.
// Backward, with g = R^T dy (. w), xh = x r and r the reciprocal norm:
//   dx = r (g - xh c),  c = sum(g xh) (L2; 0 where |x| <= eps) or mean(g xh) (RMS),
//   dw = sum over rows of (R^T dy) xh.
//
// Bound by HBM: each element is read once and written once. L lanes hold one
// row, 8 adjacent elements each (16-byte loads), so the norm is log2 L
// shuffles and the half layout's partner one shuffle. A group of L lanes stays
// on one token and walks its heads, so the 8 cosines and sines of a lane are
// read once per token; the block computes them once per token and pair into
// shared memory.
//
// Angles: the turn pos * f / (2 pi) mod 1 is an exact integer product mod 2^64
// with f / (2 pi) held as a 64-bit binary fraction, so positions of any size
// lose nothing; only the reduced turn is rounded to fp32.
#include <type_traits>

#include "layer_common.cuh"

namespace gdr {

constexpr int kNormThreads = 256;
constexpr int kNormMaxParts = 148 * 4;  // blocks that keep weight-gradient sums

struct NormArgs {
    const void *q, *k, *qw, *kw, *pos;
    const float* inv_freq;
    void *q_out, *k_out;            // forward outputs, or fp32 gradients of q and k
    const void *gq, *gk;            // backward: gradients of the outputs
    float* part;                    // backward: weight-gradient partials [blocks][2][d], or null
    long long qs[3], ks[3], gqs[3], gks[3], ps[2];
    long long tokens;
    int T, Hq, Hk, d, rot, tpb, rms, interleaved, pos64, w_f32;
    float eps, q_scale, rscale;
};

// cos and sin (times rscale) of the pairs of `tpb` tokens from token tok0.
__device__ __forceinline__ void fill_turns(const NormArgs& a, long long tok0, float* cs, float* sn) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < a.tpb * half; i += kNormThreads) {
        const int tk = i / half, p = i - tk * half;
        const long long tok = tok0 + tk;
        float c = 1.f, s = 0.f;
        if (tok < a.tokens) {
            const long long b = tok / a.T, t = tok - b * a.T;
            long long pos = t;
            if (a.pos) {
                const long long o = b * a.ps[0] + t * a.ps[1];
                pos = a.pos64 ? reinterpret_cast<const long long*>(a.pos)[o] : reinterpret_cast<const int*>(a.pos)[o];
            }
            double f = (double)a.inv_freq[p] * 0.15915494309189535;  // turns per position
            f -= floor(f);
            const unsigned long long frac = (unsigned long long)(f * 18446744073709551616.0);
            const long long turn = (long long)((unsigned long long)pos * frac);
            sincospif((float)turn * 0x1p-63f, &s, &c);
        }
        cs[i] = c * a.rscale;
        sn[i] = s * a.rscale;
    }
}

// One lane's 8 elements of a row: e(i) = 8 li + i (VEC), or li + 32 i.
template <bool VEC> __device__ __forceinline__ int row_elem(int li, int i) { return VEC ? 8 * li + i : li + 32 * i; }

template <typename T, bool VEC>
__device__ __forceinline__ void load_lane(float (&f)[8], const T* row, int li, int d) {
    if constexpr (VEC) {
        if (8 * li < d) VecIO<T, 8>::load(f, row + 8 * li);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = li + 32 * i < d ? to_f32(row[li + 32 * i]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_lane(T* row, const float (&f)[8], int li, int d) {
    if constexpr (VEC) {
        if (8 * li < d) VecIO<T, 8>::store(row + 8 * li, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (li + 32 * i < d) row[li + 32 * i] = from_f32<T>(f[i]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void load_weight(float (&w)[8], const void* p, int w_f32, int li, int d) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
        return;
    }
    if (w_f32) load_lane<float, VEC>(w, reinterpret_cast<const float*>(p), li, d);
    else load_lane<T, VEC>(w, reinterpret_cast<const T*>(p), li, d);
}

template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// c[i], s[i] of a lane's elements: out = y c + partner s (s carries the sign).
template <bool VEC>
__device__ __forceinline__ void lane_turns(float (&c)[8], float (&s)[8], const NormArgs& a, const float* cs,
                                           const float* sn, int li) {
    const int half = a.rot / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = row_elem<VEC>(li, i);
        c[i] = 1.f;
        s[i] = 0.f;
        if (e < a.rot) {
            const int p = a.interleaved ? e >> 1 : (e < half ? e : e - half);
            const bool second = a.interleaved ? (e & 1) : e >= half;
            c[i] = cs[p];
            s[i] = second ? sn[p] : -sn[p];
        }
    }
}

// The rotation's partner of each of a lane's elements. buf: this warp's row
// in shared memory (plain form only).
template <int L, bool VEC>
__device__ __forceinline__ void partners(float (&o)[8], const float (&y)[8], const NormArgs& a, int li, float* buf) {
    if constexpr (VEC) {
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = y[i ^ 1];
        } else {
            const int hv = a.rot / 16;  // vectors in half the rotated part
            const int src = li < hv ? li + hv : li < 2 * hv ? li - hv : li;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], src, L);
        }
    } else {
        const int half = a.rot / 2;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) buf[li + 32 * i] = y[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = li + 32 * i;
            o[i] = e < a.rot ? buf[a.interleaved ? e ^ 1 : (e < half ? e + half : e - half)] : 0.f;
        }
    }
}

// Reciprocal norm; `inside` tells an L2 row at or below eps (constant divisor).
__device__ __forceinline__ float row_rnorm(const NormArgs& a, float ss, bool* inside) {
    if (a.rms) {
        *inside = false;
        return rsqrtf(ss / (float)a.d + a.eps);
    }
    const float r = rsqrtf(ss), lim = 1.f / a.eps;
    *inside = r >= lim;  // a NaN row stays NaN
    return *inside ? lim : r;
}

template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(kNormThreads) qk_norm_fwd_kernel(NormArgs a) {
    extern __shared__ float sm[];
    __shared__ float rowbuf[VEC ? 1 : kNormThreads / 32][VEC ? 1 : 256];
    constexpr int kSlots = kNormThreads / L, kAhead = 4;
    float *cs = sm, *sn = sm + a.tpb * (a.rot / 2);
    const int li = threadIdx.x % L, slot = threadIdx.x / L;
    const int spt = kSlots / a.tpb;  // lane groups that share a token
    const long long tok0 = (long long)blockIdx.x * a.tpb, tok = tok0 + slot / spt;
    const int R = a.Hq + a.Hk;
    if (a.rot) {
        fill_turns(a, tok0, cs, sn);
        __syncthreads();
    }
    float c[8], s[8], qw[8], kw[8];
    lane_turns<VEC>(c, s, a, cs + (slot / spt) * (a.rot / 2), sn + (slot / spt) * (a.rot / 2), li);
    load_weight<T, VEC>(qw, a.qw, a.w_f32, li, a.d);
    load_weight<T, VEC>(kw, a.kw, a.w_f32, li, a.d);
    const bool live = tok < a.tokens;
    const long long b = live ? tok / a.T : 0, t = live ? tok - b * a.T : 0;
    const T* qrow = reinterpret_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1];
    const T* krow = reinterpret_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1];
    float* buf = rowbuf[VEC ? 0 : slot];
    // every lane of a warp runs the same number of rows: shuffles need them all
    for (int h0 = 0; h0 < R; h0 += kAhead * spt) {
        float x[kAhead][8];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int h = h0 + j * spt + slot % spt;
            if (live && h < R)
                load_lane<T, VEC>(x[j], h < a.Hq ? qrow + h * a.qs[2] : krow + (h - a.Hq) * a.ks[2], li, a.d);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int h = h0 + j * spt + slot % spt;
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[j][i], x[j][i], ss);
            bool inside;
            const float r = row_rnorm(a, row_sum<L>(ss), &inside);
            const bool isq = h < a.Hq;
            float y[8], o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[j][i] * r * (isq ? qw[i] : kw[i]);
            if (a.rot) {
                partners<L, VEC>(o, y, a, li, buf);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = s[i] == 0.f ? y[i] * c[i] : fmaf(o[i], s[i], y[i] * c[i]);
            }
            if (isq)
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= a.q_scale;
            if (live && h < R) {
                T* out = isq ? reinterpret_cast<T*>(a.q_out) + (tok * a.Hq + h) * a.d
                             : reinterpret_cast<T*>(a.k_out) + (tok * a.Hk + (h - a.Hq)) * a.d;
                store_lane<T, VEC>(out, y, li, a.d);
            }
        }
    }
}

template <typename T, typename TG, int L, bool VEC>
__global__ void __launch_bounds__(kNormThreads) qk_norm_bwd_kernel(NormArgs a) {
    extern __shared__ float sm[];
    __shared__ float rowbuf[VEC ? 1 : kNormThreads / 32][VEC ? 1 : 256];
    constexpr int kSlots = kNormThreads / L, kAhead = 2;
    float *cs = sm, *sn = sm + a.tpb * (a.rot / 2);
    const int li = threadIdx.x % L, slot = threadIdx.x / L;
    const int spt = kSlots / a.tpb;
    const int R = a.Hq + a.Hk;
    float qw[8], kw[8], dqw[8], dkw[8];
    load_weight<T, VEC>(qw, a.qw, a.w_f32, li, a.d);
    load_weight<T, VEC>(kw, a.kw, a.w_f32, li, a.d);
#pragma unroll
    for (int i = 0; i < 8; ++i) dqw[i] = dkw[i] = 0.f;
    float* buf = rowbuf[VEC ? 0 : slot];
    for (long long tok0 = (long long)blockIdx.x * a.tpb; tok0 < a.tokens; tok0 += (long long)gridDim.x * a.tpb) {
        const long long tok = tok0 + slot / spt;
        if (a.rot) {
            __syncthreads();
            fill_turns(a, tok0, cs, sn);
            __syncthreads();
        }
        float c[8], s[8];
        lane_turns<VEC>(c, s, a, cs + (slot / spt) * (a.rot / 2), sn + (slot / spt) * (a.rot / 2), li);
        const bool live = tok < a.tokens;
        const long long b = live ? tok / a.T : 0, t = live ? tok - b * a.T : 0;
        const T* qrow = reinterpret_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1];
        const T* krow = reinterpret_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1];
        const TG* gqrow = reinterpret_cast<const TG*>(a.gq) + b * a.gqs[0] + t * a.gqs[1];
        const TG* gkrow = reinterpret_cast<const TG*>(a.gk) + b * a.gks[0] + t * a.gks[1];
        for (int h0 = 0; h0 < R; h0 += kAhead * spt) {
            float x[kAhead][8], g[kAhead][8];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int h = h0 + j * spt + slot % spt;
                if (live && h < R) {
                    load_lane<T, VEC>(x[j], h < a.Hq ? qrow + h * a.qs[2] : krow + (h - a.Hq) * a.ks[2], li, a.d);
                    load_lane<TG, VEC>(g[j], h < a.Hq ? gqrow + h * a.gqs[2] : gkrow + (h - a.Hq) * a.gks[2], li, a.d);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j][i] = g[j][i] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int h = h0 + j * spt + slot % spt;
                const bool isq = h < a.Hq, on = live && h < R;
                if (isq)
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[j][i] *= a.q_scale;
                if (a.rot) {  // R^T: the partner's coefficient is -s
                    float o[8];
                    partners<L, VEC>(o, g[j], a, li, buf);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        g[j][i] = s[i] == 0.f ? g[j][i] * c[i] : fmaf(-o[i], s[i], g[j][i] * c[i]);
                }
                float ss = 0.f, gx = 0.f, gw[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    gw[i] = g[j][i] * (isq ? qw[i] : kw[i]);
                    ss = fmaf(x[j][i], x[j][i], ss);
                    gx = fmaf(gw[i], x[j][i], gx);
                }
                bool inside;
                const float r = row_rnorm(a, row_sum<L>(ss), &inside);
                gx = row_sum<L>(gx) * r;  // sum(g xh)
                const float m = inside ? 0.f : a.rms ? gx / (float)a.d : gx;
                float dx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = x[j][i] * r;
                    dx[i] = r * fmaf(-xh, m, gw[i]);
                    if (on) {
                        if (isq) dqw[i] = fmaf(g[j][i], xh, dqw[i]);
                        else dkw[i] = fmaf(g[j][i], xh, dkw[i]);
                    }
                }
                if (on) {
                    float* out = isq ? reinterpret_cast<float*>(a.q_out) + (tok * a.Hq + h) * a.d
                                     : reinterpret_cast<float*>(a.k_out) + (tok * a.Hk + (h - a.Hq)) * a.d;
                    store_lane<float, VEC>(out, dx, li, a.d);
                }
            }
        }
    }
    if (!a.part) return;
    // the block's weight gradients: lane groups added in order
    __shared__ float red[kSlots][L * 8];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) red[slot][row_elem<VEC>(li, i)] = which ? dkw[i] : dqw[i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.d; e += kNormThreads) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) v += red[k][e];
            a.part[((size_t)blockIdx.x * 2 + which) * a.d + e] = v;
        }
    }
}

// dq_weight, dk_weight [d]: 32 columns x 8 slices of the blocks' partials.
__global__ void __launch_bounds__(256) qk_norm_reduce_kernel(const float* __restrict__ part, float* __restrict__ dqw,
                                                             float* __restrict__ dkw, int parts, int d) {
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    __shared__ float sm[8][32];
    float a = 0.f;
    dependent_wait();
    if (col < 2 * d)
        for (int p = sl; p < parts; p += 8) a += part[(size_t)p * 2 * d + col];
    sm[sl][lane] = a;
    __syncthreads();
    if (sl == 0 && col < 2 * d) {
#pragma unroll
        for (int k = 1; k < 8; ++k) a += sm[k][lane];
        if (col < d) { if (dqw) dqw[col] = a; }
        else if (dkw) dkw[col - d] = a;
    }
}

// Lanes of a row: a power of two that covers d / 8 vectors; 32 in the plain form.
static int norm_lanes(int d) {
    int l = 2;
    while (l * 8 < d) l *= 2;
    return l;
}

// Tokens per block: one per lane group when that still gives every SM four
// blocks, fewer (several groups share a token's heads) below that.
static int norm_tokens_per_block(long long tokens, int lanes) {
    int tpb = kNormThreads / lanes;
    while (tpb > 1 && (tokens + tpb - 1) / tpb < 148 * 4) tpb /= 2;
    return tpb < 16 ? tpb : 16;
}

template <typename F> static void dispatch_lanes(bool vec, int lanes, F&& f) {
    if (!vec) { f(std::integral_constant<int, 32>(), std::false_type()); return; }
    switch (lanes) {
        case 2: f(std::integral_constant<int, 2>(), std::true_type()); break;
        case 4: f(std::integral_constant<int, 4>(), std::true_type()); break;
        case 8: f(std::integral_constant<int, 8>(), std::true_type()); break;
        case 16: f(std::integral_constant<int, 16>(), std::true_type()); break;
        default: f(std::integral_constant<int, 32>(), std::true_type()); break;
    }
}

static gdr_status norm_fill(NormArgs& a, const long long* strides, int nstrides, const void* q, const void* k,
                            const void* qw, const void* kw, const void* pos, const float* inv_freq, int B, int T,
                            int Hq, int Hk, int d, int rot, int kind, int rotary, float eps, float q_scale,
                            float rscale, int pos64, int dtype, int weight_dtype) {
    if (B < 1 || T < 0 || Hq < 1 || Hk < 0 || d < 1 || rot < 0 || !dtype_ok(dtype) || !dtype_ok(weight_dtype))
        return GDR_ERR_INVALID_ARG;
    if (kind != GDR_NORM_L2 && kind != GDR_NORM_RMS) return GDR_ERR_INVALID_ARG;
    if (rotary != GDR_ROTARY_HALF && rotary != GDR_ROTARY_INTERLEAVED) return GDR_ERR_INVALID_ARG;
    if (!(eps > 0.f)) return GDR_ERR_INVALID_ARG;
    if (kind == GDR_NORM_L2 && (qw || kw)) return GDR_ERR_INVALID_ARG;
    if (rot % 2 || rot > d || (rot > 0) != (inv_freq != nullptr) || (pos && !rot)) return GDR_ERR_INVALID_ARG;
    if (pos64 != 0 && pos64 != 1) return GDR_ERR_INVALID_ARG;
    if ((Hk > 0) != (k != nullptr) && T > 0) return GDR_ERR_INVALID_ARG;
    if ((Hk == 0 && kw) || (T > 0 && !q)) return GDR_ERR_INVALID_ARG;
    if (d > 256) return GDR_ERR_UNSUPPORTED;
    if (weight_dtype != dtype && weight_dtype != GDR_FP32) return GDR_ERR_UNSUPPORTED;
    const size_t e = dtype_size(dtype), ew = dtype_size(weight_dtype);
    if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(qw, ew) || !aligned_to(kw, ew) ||
        !aligned_to(inv_freq, 4) || !aligned_to(pos, pos64 ? 8 : 4))
        return GDR_ERR_MISALIGNED;
    a = NormArgs{};
    a.q = q; a.k = k; a.qw = qw; a.kw = kw; a.pos = pos; a.inv_freq = inv_freq;
    a.tokens = (long long)B * T;
    a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot;
    a.rms = kind == GDR_NORM_RMS; a.interleaved = rotary == GDR_ROTARY_INTERLEAVED;
    a.pos64 = pos64; a.w_f32 = weight_dtype == GDR_FP32;
    a.eps = eps; a.q_scale = q_scale; a.rscale = rscale;
    const long long dense[14] = {(long long)T * Hq * d, (long long)Hq * d, d, (long long)T * Hk * d, (long long)Hk * d, d,
                                 T, 1, (long long)T * Hq * d, (long long)Hq * d, d, (long long)T * Hk * d,
                                 (long long)Hk * d, d};
    const long long* s = strides ? strides : dense;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = s[i];
        a.ks[i] = s[3 + i];
        if (nstrides == 14) { a.gqs[i] = s[8 + i]; a.gks[i] = s[11 + i]; }
    }
    a.ps[0] = s[6]; a.ps[1] = s[7];
    return GDR_OK;
}

// The 16-byte form: rows of whole 8-element vectors, every stride a multiple
// of 8, every pointer 16-byte aligned, and half-layout partners in whole vectors.
static bool norm_vector(const NormArgs& a, bool bwd, size_t eg) {
    if (a.d % 8) return false;
    if (a.rot && !a.interleaved && a.rot % 16) return false;
    for (const void* p : {a.q, a.k, a.qw, a.kw, (const void*)a.q_out, (const void*)a.k_out, a.gq, a.gk})
        if (!aligned_to(p, 16)) return false;
    for (int i = 0; i < 3; ++i)
        if (a.qs[i] % 8 || a.ks[i] % 8 || (bwd && (a.gqs[i] % 8 || a.gks[i] % 8))) return false;
    (void)eg;
    return true;
}

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_qk_norm_fwd(const void* q, const void* k, const void* q_weight, const void* k_weight,
                           const void* positions, const float* inv_freq, void* q_out, void* k_out,
                           const long long* strides, int B, int T, int H_q, int H_k, int d, int rot, int kind,
                           int rotary, float eps, float q_scale, float rotary_scale, int position_int64, int dtype,
                           int weight_dtype, void* stream) {
    NormArgs a;
    gdr_status ok = norm_fill(a, strides, 8, q, k, q_weight, k_weight, positions, inv_freq, B, T, H_q, H_k, d, rot,
                              kind, rotary, eps, q_scale, rotary_scale, position_int64, dtype, weight_dtype);
    if (ok != GDR_OK) return ok;
    if (T == 0) return GDR_OK;
    if (!q_out || (H_k > 0) != (k_out != nullptr)) return GDR_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned_to(q_out, e) || !aligned_to(k_out, e)) return GDR_ERR_MISALIGNED;
    a.q_out = q_out; a.k_out = k_out;
    const bool vec = norm_vector(a, false, e);
    const int lanes = vec ? norm_lanes(d) : 32;
    a.tpb = norm_tokens_per_block(a.tokens, lanes);
    const long long grid = (a.tokens + a.tpb - 1) / a.tpb;
    if (grid > 0x7fffffffll) return GDR_ERR_UNSUPPORTED;
    const size_t smem = (size_t)a.tpb * rot * sizeof(float);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    dispatch_lanes(vec, lanes, [&](auto lc, auto vc) {
        constexpr int L = decltype(lc)::value;
        constexpr bool V = decltype(vc)::value;
        if (dtype == GDR_BF16) qk_norm_fwd_kernel<__nv_bfloat16, L, V><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
        else qk_norm_fwd_kernel<float, L, V><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
    });
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

size_t gdr_qk_norm_bwd_workspace_size(int d) {
    return d < 1 ? 0 : round256((size_t)kNormMaxParts * 2 * d * sizeof(float));
}

gdr_status gdr_qk_norm_bwd(const void* q, const void* k, const void* q_weight, const void* k_weight,
                           const void* positions, const float* inv_freq, const void* dq_out, const void* dk_out,
                           float* dq, float* dk, float* dq_weight, float* dk_weight, void* workspace,
                           size_t workspace_bytes, const long long* strides, int B, int T, int H_q, int H_k, int d,
                           int rot, int kind, int rotary, float eps, float q_scale, float rotary_scale,
                           int position_int64, int dtype, int weight_dtype, int grad_dtype, void* stream) {
    NormArgs a;
    gdr_status ok = norm_fill(a, strides, 14, q, k, q_weight, k_weight, positions, inv_freq, B, T, H_q, H_k, d, rot,
                              kind, rotary, eps, q_scale, rotary_scale, position_int64, dtype, weight_dtype);
    if (ok != GDR_OK) return ok;
    if (!dtype_ok(grad_dtype)) return GDR_ERR_INVALID_ARG;
    if (grad_dtype != dtype && grad_dtype != GDR_FP32) return GDR_ERR_UNSUPPORTED;
    if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr))
        return GDR_ERR_INVALID_ARG;
    if (T > 0 && (!dq_out || !dq || (H_k > 0) != (dk_out != nullptr) || (H_k > 0) != (dk != nullptr)))
        return GDR_ERR_INVALID_ARG;
    const size_t eg = dtype_size(grad_dtype);
    if (!aligned_to(dq_out, eg) || !aligned_to(dk_out, eg) || !aligned_to(dq, 4) || !aligned_to(dk, 4) ||
        !aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4))
        return GDR_ERR_MISALIGNED;
    const bool weights = q_weight || k_weight;
    if (weights) {
        if (!workspace || workspace_bytes < gdr_qk_norm_bwd_workspace_size(d)) return GDR_ERR_INVALID_ARG;
        if (!aligned_to(workspace, 256)) return GDR_ERR_MISALIGNED;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    a.gq = dq_out; a.gk = dk_out;
    a.q_out = dq; a.k_out = dk;
    a.part = weights ? reinterpret_cast<float*>(workspace) : nullptr;
    long long grid = 0;
    if (T > 0) {
        const bool vec = norm_vector(a, true, eg);
        const int lanes = vec ? norm_lanes(d) : 32;
        a.tpb = norm_tokens_per_block(a.tokens, lanes);
        grid = (a.tokens + a.tpb - 1) / a.tpb;
        if (grid > kNormMaxParts) grid = kNormMaxParts;
        const size_t smem = (size_t)a.tpb * rot * sizeof(float);
        dispatch_lanes(vec, lanes, [&](auto lc, auto vc) {
            constexpr int L = decltype(lc)::value;
            constexpr bool V = decltype(vc)::value;
            if (dtype == GDR_FP32)
                qk_norm_bwd_kernel<float, float, L, V><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
            else if (grad_dtype == GDR_FP32)
                qk_norm_bwd_kernel<__nv_bfloat16, float, L, V><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
            else
                qk_norm_bwd_kernel<__nv_bfloat16, __nv_bfloat16, L, V><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
        });
        if (cudaGetLastError() != cudaSuccess) return GDR_ERR_LAUNCH;
    }
    if (!weights) return GDR_OK;
    return launch_dependent(qk_norm_reduce_kernel, (unsigned)((2 * d + 31) / 32), 256, 0, st, a.part, dq_weight,
                            dk_weight, (int)grid, d) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

}  // extern "C"
