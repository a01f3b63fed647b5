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
// shuffles and the half layout's partner one shuffle per element. A group of L
// lanes stays on one token and walks its heads, so a lane's 8 cosines and sines
// are read once per token; the block computes them once per token and pair into
// shared memory, with the first rows already requested. The first version came
// to 30% of the copy rate: 27 instructions an element, most of them copies,
// clearing and layout tests; reloading a row's registers as soon as it is
// unpacked and a kernel per layout brought it to 86%.
//
// Angles: the turn pos * f / (2 pi) mod 1 is an exact integer product mod 2^64
// with f / (2 pi), computed in 64-bit floating point, as a binary fraction; only
// the reduced turn is rounded to fp32.
#include <type_traits>

#include "layer_common.cuh"

namespace gdr {

// Rows a lane group requests ahead, and blocks per SM. Forward, 2 x 8192 tokens
// of 64 heads of 128 in bf16 (94 us, 5.7 TB/s): 4 and 3; 2 and 3 took 1.11 times
// as long, 2 and 4 and 4 and 4 (spills) 1.08 times. Backward, 2 x 4096 tokens of
// 32 heads of 256 (109 us, 4.9 TB/s): 3 and 2; 2 and 2 1.02 times, 1 and 2 and 1
// and 3 (spills) about 1.2 times.
constexpr int kFwdAhead = 4, kFwdBlocks = 3, kBwdAhead = 3, kBwdBlocks = 2;
constexpr int kNormThreads = 256;
constexpr int kNormMaxParts = 148 * kBwdBlocks;  // backward: one wave of blocks, each with sums of its own

struct NormArgs {
    const void *q, *k, *qw, *kw, *pos;
    const float* inv_freq;
    void *q_out, *k_out;            // forward outputs, or fp32 gradients of q and k
    const void *gq, *gk;            // backward: gradients of the outputs
    float* part;                    // backward: weight-gradient partials [blocks][2][d], or null
    long long qs[3], ks[3], gqs[3], gks[3], ps[2];
    long long tokens;
    int T, Hq, Hk, d, rot, tpb, rms, interleaved, pos64, w_f32, pairs;
    float eps, q_scale, rscale, inv_d, inv_eps;
};

// ROT: layout of the rotation, 0 for none. kHalfShared: partners that do not lie
// in whole vectors (rot not a multiple of 16) go through shared memory.
enum { kHalf = 1, kInterleaved = 2, kHalfShared = 3 };

// Sequence and position in it of a token.
__device__ __forceinline__ void token_of(const NormArgs& a, long long tok, long long& b, long long& t) {
    b = a.tokens <= 0x7fffffff ? (unsigned)tok / (unsigned)a.T : tok / a.T;
    t = tok - b * a.T;
}

// What the turns of a block's tokens are made of: each pair's turns per position
// as a binary fraction, and the tokens' positions.
struct TurnParts {
    unsigned long long frac[128];
    long long pos[16];
};
__device__ __forceinline__ void fill_frequencies(TurnParts& tp, const NormArgs& a) {
    for (int p = threadIdx.x; p < a.rot / 2; p += kNormThreads) {
        double f = (double)a.inv_freq[p] * 0.15915494309189535;  // 1 / (2 pi)
        f -= floor(f);
        tp.frac[p] = (unsigned long long)(f * 18446744073709551616.0);
    }
}
__device__ __forceinline__ void fill_positions(TurnParts& tp, const NormArgs& a, long long tok0) {
    const int i = kNormThreads - 1 - threadIdx.x;  // threads that the frequencies leave free
    const long long tok = tok0 + i;
    if (i >= a.tpb || tok >= a.tokens) return;
    long long b, t;
    token_of(a, tok, b, t);
    if (a.pos) {
        const long long o = b * a.ps[0] + t * a.ps[1];
        t = a.pos64 ? reinterpret_cast<const long long*>(a.pos)[o] : reinterpret_cast<const int*>(a.pos)[o];
    }
    tp.pos[i] = t;
}
// cos and sin (times rscale) of the pairs of `tpb` tokens from token tok0.
__device__ __forceinline__ void fill_turns(const TurnParts& tp, const NormArgs& a, long long tok0, float* cs, float* sn) {
    const unsigned half = a.rot / 2;
    for (unsigned i = threadIdx.x; i < a.tpb * half; i += kNormThreads) {
        const unsigned tk = i / half, p = i - tk * half;
        float c = 1.f, s = 0.f;
        if (tok0 + tk < a.tokens) {
            const long long turn = (long long)((unsigned long long)tp.pos[tk] * tp.frac[p]);
            sincospif((float)turn * 0x1p-63f, &s, &c);
        }
        cs[i] = c * a.rscale;
        sn[i] = s * a.rscale;
    }
}

// One lane's 8 elements of a row: 8 li + i (VEC), or the pairs li + L j.
template <int L, bool VEC> __device__ __forceinline__ int row_elem(int li, int i) { return VEC ? 8 * li + i : 2 * (li + L * (i >> 1)) + (i & 1); }

// The elements as loaded, and as numbers. A lane's elements from d on are
// never loaded and stay 0; a row that is not wanted keeps what it held.
template <typename T, int L, bool VEC> struct LaneRow {
    RawVec<T, 8> v;
    __device__ __forceinline__ void load(const T* row, int li, int d, bool on, int pairs) {
        if constexpr (VEC) {
            if (on) v.load(row);
        } else if (pairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                RawVec<T, 2> p;
                if (!on || row_elem<L, VEC>(li, 2 * j) >= d) continue;
                p.load(row + 2 * L * j);
#pragma unroll
                for (int i = 0; i < RawVec<T, 2>::kWords; ++i) v.w[RawVec<T, 2>::kWords * j + i] = p.w[i];
            }
        } else {
            if (on) v.zero();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (on && row_elem<L, VEC>(li, i) < d) v.set(i, row[row_elem<L, VEC>(0, i)]);
        }
    }
    __device__ __forceinline__ void get(f2 (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pack2(v.get(2 * i), v.get(2 * i + 1));
    }
};
template <typename T, int L, bool VEC>
__device__ __forceinline__ void store_lane(T* row, const f2 (&v)[4], int li, int d, int pairs) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    if constexpr (VEC) {
        VecIO<T, 8>::store(row, f);
    } else if (pairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row_elem<L, VEC>(li, 2 * j) < d) VecIO<T, 2>::store(row + 2 * L * j, f + 2 * j);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row_elem<L, VEC>(li, i) < d) row[row_elem<L, VEC>(0, i)] = from_f32<T>(f[i]);
    }
}

// q's and k's weights as fp32 in shared memory, rows of 256: ones where absent,
// zeros from d on. Lanes read past d, and their elements there enter the row's
// sums as 0 * weight, so what an earlier kernel left (NaN) must not stay.
template <typename T> __device__ __forceinline__ void fill_weights(float* sw, const NormArgs& a, float q_scale) {
    for (int i = threadIdx.x; i < 512; i += kNormThreads) {
        const int e = i & 255;
        const bool isq = i < 256;
        const void* p = isq ? a.qw : a.kw;
        float w = 0.f;
        if (e < a.d) w = !p ? 1.f : a.w_f32 ? reinterpret_cast<const float*>(p)[e] : to_f32(reinterpret_cast<const T*>(p)[e]);
        sw[i] = isq ? w * q_scale : w;
    }
}
template <int L, bool VEC> __device__ __forceinline__ void lane_weight(f2 (&w)[4], const float* sw, int li) {
    float f[8];
    if constexpr (VEC) {
        VecIO<float, 8>::load(f, sw + 8 * li);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = sw[row_elem<L, VEC>(li, i)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1]);
}

template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// c, s of a lane's elements: out = y c + partner s (s carries the sign, and
// another for the transposed rotation: sign = -1); 1 and 0 where not rotated.
template <int L, bool VEC, int ROT>
__device__ __forceinline__ void lane_turns(f2 (&c)[4], f2 (&s)[4], const NormArgs& a, const float* cs, const float* sn,
                                           int li, float sign) {
    const int half = a.rot / 2;
    float cf[8], sf[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = row_elem<L, VEC>(li, i);
        cf[i] = 1.f;
        sf[i] = 0.f;
        if (e < a.rot) {
            const int p = ROT == kInterleaved ? e >> 1 : (e < half ? e : e - half);
            const bool second = ROT == kInterleaved ? (e & 1) : e >= half;
            cf[i] = cs[p];
            sf[i] = second ? sign * sn[p] : -sign * sn[p];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = pack2(cf[2 * i], cf[2 * i + 1]);
        s[i] = pack2(sf[2 * i], sf[2 * i + 1]);
    }
}

// Turns a lane's elements in place. src: the lane of the half layout's
// partners (its own where not rotated). buf: the lane group's row in shared
// memory (kHalfShared, and kHalf of the plain form).
template <int L, bool VEC, int ROT>
__device__ __forceinline__ void rotate(f2 (&y)[4], const f2 (&c)[4], const f2 (&s)[4], const NormArgs& a, int li,
                                       int src, float* buf) {
    float f[8], o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(y[i], f[2 * i], f[2 * i + 1]);
    if constexpr (ROT == kInterleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f[i ^ 1];
    } else if constexpr (VEC && ROT == kHalf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, f[i], src, L);
    } else {
        const int half = a.rot / 2;
        __syncwarp();
        if constexpr (VEC) {
            VecIO<float, 8>::store(buf + 8 * li, f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) buf[row_elem<L, VEC>(li, i)] = f[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = row_elem<L, VEC>(li, i);
            o[i] = e < a.rot ? buf[e < half ? e + half : e - half] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fma2(pack2(o[2 * i], o[2 * i + 1]), s[i], mul2(y[i], c[i]));
}

// The lane that holds the half layout's partners of a lane's elements.
__device__ __forceinline__ int partner_lane(const NormArgs& a, int li) {
    const int hv = a.rot / 16;  // vectors in half the rotated part
    return li < hv ? li + hv : li < 2 * hv ? li - hv : li;
}

// Reciprocal norm; `inside` tells an L2 row at or below eps (constant divisor).
__device__ __forceinline__ float row_rnorm(const NormArgs& a, float ss, bool* inside) {
    if (a.rms) {
        *inside = false;
        return rsqrt_approx(fmaf(ss, a.inv_d, a.eps));
    }
    const float r = rsqrt_approx(ss);
    const float lim = a.inv_eps;
    *inside = r >= lim;  // a NaN row stays NaN
    return *inside ? lim : r;
}

// The rows of one lane group's token at this lane's first element: head h of
// q, then of k.
template <typename T> struct HeadRows {
    T *q, *k;  // k is reached from h = 0 too, H_q heads before its first
    long long qs, ks;
    int Hq;
    __device__ __forceinline__ HeadRows(T* q_, T* k_, long long qs_, long long ks_, int Hq_)
        : q(q_), k(k_ - Hq_ * ks_), qs(qs_), ks(ks_), Hq(Hq_) {}
    __device__ __forceinline__ T* at(int h) const { return (h < Hq ? q : k) + h * (h < Hq ? qs : ks); }
};
template <typename T>
__device__ __forceinline__ HeadRows<const T> input_rows(const void* q, const void* k, const long long (&qs)[3],
                                                        const long long (&ks)[3], long long b, long long t, int Hq,
                                                        int e0) {
    return {reinterpret_cast<const T*>(q) + b * qs[0] + t * qs[1] + e0,
            reinterpret_cast<const T*>(k) + b * ks[0] + t * ks[1] + e0, qs[2], ks[2], Hq};
}
template <typename T>
__device__ __forceinline__ HeadRows<T> output_rows(void* q, void* k, long long tok, int Hq, int Hk, int d, int e0) {
    return {reinterpret_cast<T*>(q) + tok * Hq * d + e0, reinterpret_cast<T*>(k) + tok * Hk * d + e0, d, d, Hq};
}

template <typename T, int L, bool VEC, int ROT>
__global__ void __launch_bounds__(kNormThreads, kFwdBlocks) qk_norm_fwd_kernel(NormArgs a) {
    extern __shared__ float sm[];
    constexpr bool kBuf = (!VEC && ROT == kHalf) || ROT == kHalfShared;
    __shared__ __align__(16) float rowbuf[kBuf ? kNormThreads / L : 1][kBuf ? 8 * L : 1];
    __shared__ __align__(16) float sw[512];
    constexpr int kSlots = kNormThreads / L, kAhead = sizeof(T) == 2 ? kFwdAhead : kFwdAhead / 2;
    float *cs = sm, *sn = sm + a.tpb * (a.rot / 2);
    const int li = threadIdx.x % L, slot = threadIdx.x / L, e0 = row_elem<L, VEC>(li, 0);
    const int spt = kSlots / a.tpb;  // lane groups that share a token
    const long long tok0 = (long long)blockIdx.x * a.tpb, tok = tok0 + slot / spt;
    const int R = a.Hq + a.Hk, h0 = slot % spt, src = partner_lane(a, li);
    const bool live = tok < a.tokens && e0 < a.d, weighted = a.qw || a.kw;
    long long b, t;
    token_of(a, live ? tok : 0, b, t);
    const int last = live ? R : 0;  // this lane's rows end here
    const auto in = input_rows<T>(a.q, a.k, a.qs, a.ks, b, t, a.Hq, e0);
    const auto out = output_rows<T>(a.q_out, a.k_out, tok, a.Hq, a.Hk, a.d, e0);
    dependent_launch();
    dependent_wait();
    LaneRow<T, L, VEC> row[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        row[j].v.zero();
        row[j].load(in.at(h0 + j * spt), li, a.d, h0 + j * spt < last, a.pairs);
    }
    if (weighted) fill_weights<T>(sw, a, a.q_scale);
    if constexpr (ROT != 0) {
        __shared__ TurnParts tp;
        fill_frequencies(tp, a);
        fill_positions(tp, a, tok0);
        __syncthreads();
        fill_turns(tp, a, tok0, cs, sn);
    }
    if (weighted || ROT) __syncthreads();
    f2 c[4], s[4];
    if (ROT) lane_turns<L, VEC, ROT>(c, s, a, cs + (slot / spt) * (a.rot / 2), sn + (slot / spt) * (a.rot / 2), li, 1.f);
    float* buf = rowbuf[kBuf ? slot : 0];
    // every lane of a warp runs the same number of rows: shuffles need them all
    for (int hb = 0; hb < R; hb += kAhead * spt) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int h = hb + h0 + j * spt, ahead = h + kAhead * spt;
            f2 y[4];
            row[j].get(y);
            row[j].load(in.at(ahead), li, a.d, ahead < last, a.pairs);
            f2 sq = mul2(y[0], y[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) sq = fma2(y[i], y[i], sq);
            bool inside;
            float r = row_rnorm(a, row_sum<L>(sum2(sq)), &inside);
            if (weighted) {
                f2 w[4];
                lane_weight<L, VEC>(w, sw + (h < a.Hq ? 0 : 256), li);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], mul2(both2(r), w[i]));
            } else {
                if (h < a.Hq) r *= a.q_scale;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], both2(r));
            }
            if constexpr (ROT != 0) rotate<L, VEC, ROT>(y, c, s, a, li, src, buf);
            if (h < last) store_lane<T, L, VEC>(out.at(h), y, li, a.d, a.pairs);
        }
    }
}

template <typename T, typename TG, int L, bool VEC, int ROT>
__global__ void __launch_bounds__(kNormThreads, kBwdBlocks) qk_norm_bwd_kernel(NormArgs a) {
    extern __shared__ float sm[];
    constexpr bool kBuf = (!VEC && ROT == kHalf) || ROT == kHalfShared;
    __shared__ __align__(16) float rowbuf[kBuf ? kNormThreads / L : 1][kBuf ? 8 * L : 1];
    __shared__ __align__(16) float sw[512];
    constexpr int kSlots = kNormThreads / L, kAhead = sizeof(T) == 2 ? kBwdAhead : 1;
    float *cs = sm, *sn = sm + a.tpb * (a.rot / 2);
    const int li = threadIdx.x % L, slot = threadIdx.x / L, e0 = row_elem<L, VEC>(li, 0);
    const int spt = kSlots / a.tpb;
    const int R = a.Hq + a.Hk, h0 = slot % spt, src = partner_lane(a, li);
    const bool weighted = a.qw || a.kw;
    f2 dqw[4], dkw[4];  // without q_scale
#pragma unroll
    for (int i = 0; i < 4; ++i) dqw[i] = dkw[i] = both2(0.f);
    if (weighted) fill_weights<T>(sw, a, 1.f);
    __shared__ TurnParts tp;
    if (ROT) fill_frequencies(tp, a);
    float* buf = rowbuf[kBuf ? slot : 0];
    LaneRow<T, L, VEC> xrow[kAhead];
    LaneRow<TG, L, VEC> grow[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        xrow[j].v.zero();
        grow[j].v.zero();
    }
    for (long long tok0 = (long long)blockIdx.x * a.tpb; tok0 < a.tokens; tok0 += (long long)gridDim.x * a.tpb) {
        const long long tok = tok0 + slot / spt;
        const bool live = tok < a.tokens && e0 < a.d;
        const int last = live ? R : 0;
        long long b, t;
        token_of(a, live ? tok : 0, b, t);
        const auto in = input_rows<T>(a.q, a.k, a.qs, a.ks, b, t, a.Hq, e0);
        const auto gin = input_rows<TG>(a.gq, a.gk, a.gqs, a.gks, b, t, a.Hq, e0);
        const auto out = output_rows<float>(a.q_out, a.k_out, tok, a.Hq, a.Hk, a.d, e0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int h = h0 + j * spt;
            xrow[j].load(in.at(h), li, a.d, h < last, a.pairs);
            grow[j].load(gin.at(h), li, a.d, h < last, a.pairs);
        }
        f2 c[4], s[4];  // of the transposed rotation
        if (ROT) fill_positions(tp, a, tok0);
        __syncthreads();  // the last tokens' turns have been read
        if (ROT) {
            fill_turns(tp, a, tok0, cs, sn);
            __syncthreads();
            lane_turns<L, VEC, ROT>(c, s, a, cs + (slot / spt) * (a.rot / 2), sn + (slot / spt) * (a.rot / 2), li, -1.f);
        }
        for (int hb = 0; hb < R; hb += kAhead * spt) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int h = hb + h0 + j * spt, ahead = h + kAhead * spt;
                const bool isq = h < a.Hq;
                f2 x[4], g[4], gw[4];
                xrow[j].get(x);
                grow[j].get(g);
                xrow[j].load(in.at(ahead), li, a.d, ahead < last, a.pairs);
                grow[j].load(gin.at(ahead), li, a.d, ahead < last, a.pairs);
                if constexpr (ROT != 0) rotate<L, VEC, ROT>(g, c, s, a, li, src, buf);
                if (weighted) {
                    lane_weight<L, VEC>(gw, sw + (isq ? 0 : 256), li);
#pragma unroll
                    for (int i = 0; i < 4; ++i) gw[i] = mul2(gw[i], g[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) gw[i] = g[i];
                }
                f2 sq = mul2(x[0], x[0]), gx2 = mul2(gw[0], x[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) {
                    sq = fma2(x[i], x[i], sq);
                    gx2 = fma2(gw[i], x[i], gx2);
                }
                bool inside;
                const float r = row_rnorm(a, row_sum<L>(sum2(sq)), &inside);
                const float gx = row_sum<L>(sum2(gx2)) * r;  // sum(g xh)
                const float m = inside ? 0.f : a.rms ? gx * a.inv_d : gx;
                const float rs = isq ? r * a.q_scale : r;
                f2 dx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = mul2(x[i], both2(r));  // xh
                    dx[i] = mul2(both2(rs), fma2(x[i], both2(-m), gw[i]));
                }
                if (h < last) {
                    if (weighted && isq) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) dqw[i] = fma2(g[i], x[i], dqw[i]);
                    } else if (weighted) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) dkw[i] = fma2(g[i], x[i], dkw[i]);
                    }
                    store_lane<float, L, VEC>(out.at(h), dx, li, a.d, a.pairs);
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
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            unpack2(which ? dkw[i] : mul2(dqw[i], both2(a.q_scale)), lo, hi);
            red[slot][row_elem<L, VEC>(li, 2 * i)] = lo;
            red[slot][row_elem<L, VEC>(li, 2 * i + 1)] = hi;
        }
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

// Lanes of a row: a power of two that covers d / 8.
static int norm_lanes(int d) {
    int l = 2;
    while (l * 8 < d) l *= 2;
    return l;
}

// Tokens per block: more of them share a block's cosines, fewer (several lane
// groups then share a token's heads) make more blocks. Least cost of waves of
// `blocks` blocks (backward: turns of that many), each the rows of a lane group
// and about four rows' time for the cosines: 6 x 391 tokens of 6 heads of 67
// backward take 45 us with one token a block, 9 with the number taken here.
static int norm_tokens_per_block(long long tokens, int lanes, int rows, long long blocks) {
    const int slots = kNormThreads / lanes;
    int best = 1;
    long long least = -1;
    for (int tpb = slots < 16 ? slots : 16; tpb >= 1; tpb /= 2) {
        const long long groups = (tokens + tpb - 1) / tpb, each = (rows + slots / tpb - 1) / (slots / tpb);
        const long long cost = (groups + blocks - 1) / blocks * (4 + each);
        if (least < 0 || cost < least) {
            least = cost;
            best = tpb;
        }
    }
    return best;
}

template <int L, bool VEC, typename F> static void dispatch_rot(const NormArgs& a, F&& f) {
    using LC = std::integral_constant<int, L>;
    using VC = std::integral_constant<bool, VEC>;
    if (!a.rot) f(LC(), VC(), std::integral_constant<int, 0>());
    else if (a.interleaved) f(LC(), VC(), std::integral_constant<int, kInterleaved>());
    else if (VEC && a.rot % 16) f(LC(), VC(), std::integral_constant<int, VEC ? kHalfShared : kHalf>());
    else f(LC(), VC(), std::integral_constant<int, kHalf>());
}
template <typename F> static void dispatch_lanes(const NormArgs& a, bool vec, int lanes, F&& f) {
    switch (lanes) {
        case 2: vec ? dispatch_rot<2, true>(a, f) : dispatch_rot<2, false>(a, f); break;
        case 4: vec ? dispatch_rot<4, true>(a, f) : dispatch_rot<4, false>(a, f); break;
        case 8: vec ? dispatch_rot<8, true>(a, f) : dispatch_rot<8, false>(a, f); break;
        case 16: vec ? dispatch_rot<16, true>(a, f) : dispatch_rot<16, false>(a, f); break;
        default: vec ? dispatch_rot<32, true>(a, f) : dispatch_rot<32, false>(a, f); break;
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
    if (d > 256 || !axes_fit({(long long)Hq + Hk})) return GDR_ERR_UNSUPPORTED;
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
    a.eps = eps < 1.17549435e-38f ? 1.17549435e-38f : eps;  // the kernels flush smaller numbers to 0
    a.q_scale = q_scale; a.rscale = rscale;
    a.inv_d = 1.f / (float)d; a.inv_eps = 1.f / a.eps;
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

// Rows of whole vectors of m elements: every stride a multiple of m, every
// pointer (types of e, eg and eo bytes: inputs, gradients, outputs) aligned to
// m elements, or 16 bytes.
static bool norm_rows_aligned(const NormArgs& a, int m, bool bwd, size_t e, size_t eg, size_t eo) {
    auto to = [&](size_t size) { return m * size < 16 ? m * size : 16; };
    if (a.d % m || !aligned_to(a.q, to(e)) || !aligned_to(a.k, to(e)) || !aligned_to(a.gq, to(eg)) ||
        !aligned_to(a.gk, to(eg)) || !aligned_to(a.q_out, to(eo)) || !aligned_to(a.k_out, to(eo)))
        return false;
    for (int i = 0; i < 3; ++i)
        if (a.qs[i] % m || a.ks[i] % m || (bwd && (a.gqs[i] % m || a.gks[i] % m))) return false;
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
    const bool vec = norm_rows_aligned(a, 8, false, e, e, e);
    a.pairs = norm_rows_aligned(a, 2, false, e, e, e);
    const int lanes = norm_lanes(d);
    a.tpb = norm_tokens_per_block(a.tokens, lanes, H_q + H_k, 148 * kFwdBlocks);
    const long long grid = (a.tokens + a.tpb - 1) / a.tpb;
    if (grid > 0x7fffffffll) return GDR_ERR_UNSUPPORTED;
    const size_t smem = (size_t)a.tpb * rot * sizeof(float);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = cudaErrorInvalidValue;
    dispatch_lanes(a, vec, lanes, [&](auto lc, auto vc, auto rc) {
        constexpr int L = decltype(lc)::value;
        constexpr bool V = decltype(vc)::value;
        constexpr int RT = decltype(rc)::value;
        err = dtype == GDR_BF16
                  ? launch_dependent(qk_norm_fwd_kernel<__nv_bfloat16, L, V, RT>, (unsigned)grid, kNormThreads, smem, st, a)
                  : launch_dependent(qk_norm_fwd_kernel<float, L, V, RT>, (unsigned)grid, kNormThreads, smem, st, a);
    });
    return err == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
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
        const size_t e = dtype_size(dtype);
        const bool vec = norm_rows_aligned(a, 8, true, e, eg, 4);
        a.pairs = norm_rows_aligned(a, 2, true, e, eg, 4);
        const int lanes = norm_lanes(d);
        a.tpb = norm_tokens_per_block(a.tokens, lanes, H_q + H_k, kNormMaxParts);
        grid = (a.tokens + a.tpb - 1) / a.tpb;
        if (grid > kNormMaxParts) grid = kNormMaxParts;
        const size_t smem = (size_t)a.tpb * rot * sizeof(float);
        dispatch_lanes(a, vec, lanes, [&](auto lc, auto vc, auto rc) {
            constexpr int L = decltype(lc)::value;
            constexpr bool V = decltype(vc)::value;
        constexpr int RT = decltype(rc)::value;
            if (dtype == GDR_FP32)
                qk_norm_bwd_kernel<float, float, L, V, RT><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
            else if (grad_dtype == GDR_FP32)
                qk_norm_bwd_kernel<__nv_bfloat16, float, L, V, RT><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
            else
                qk_norm_bwd_kernel<__nv_bfloat16, __nv_bfloat16, L, V, RT><<<(unsigned)grid, kNormThreads, smem, st>>>(a);
        });
        if (cudaGetLastError() != cudaSuccess) return GDR_ERR_LAUNCH;
    }
    if (!weights) return GDR_OK;
    return launch_dependent(qk_norm_reduce_kernel, (unsigned)((2 * d + 31) / 32), 256, 0, st, a.part, dq_weight,
                            dk_weight, (int)grid, d) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

}  // extern "C"
