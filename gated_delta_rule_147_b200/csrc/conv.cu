// Short causal depthwise convolution: forward, backward and single token.
//
// Per channel, with W taps and the W - 1 inputs before the sequence carried
// in X0 (zeros without it):
//   p_t = bias + sum_j w_j x_{t-W+1+j},   y_t = p_t sigmoid(p_t)  (or p_t),
//   X_T = the last W - 1 inputs.
// Backward, with dp_t = dy_t dy/dp (sigmoid(p)(1 + p(1 - sigmoid(p)))):
//   dx_s = sum_j w_j dp_{s+W-1-j},  dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t.
//
// Bound by HBM: a token-channel is read once and written once against about
// 2 W + 6 flops. One thread owns V adjacent channels (16-byte rows) and walks
// `tt` tokens with the last W - 1 inputs in registers, so a row is loaded once
// per chunk (plus W - 1 halo rows, which L2 serves); eight rows are requested
// before the first is used. Threads are numbered with the channel vector
// fastest, so narrow layers fill warps too. All sums are fp32; y is rounded
// once, gradients are fp32.
#include "layer_common.cuh"

namespace gdr {

constexpr int kConvBatch = 8;  // rows requested ahead of their use

struct ConvShape {
    int T, D, nvec, nchunk, tt, silu, w_f32;
    unsigned total;  // threads: B * nchunk * nvec
};

// Filter taps of V channels: [D, W] row-major is V * W consecutive elements.
template <typename T, int V, int W>
__device__ __forceinline__ void load_taps(float (&w)[W][V], float (&bias)[V], const void* weight,
                                          const void* bp, int c, int w_f32) {
    float flat[V * W];
    if (w_f32) {
        const float* p = reinterpret_cast<const float*>(weight) + (size_t)c * W;
#pragma unroll
        for (int i = 0; i < V * W; i += (V > 1 ? 4 : 1)) VecIO<float, (V > 1 ? 4 : 1)>::load(flat + i, p + i);
    } else {
        const T* p = reinterpret_cast<const T*>(weight) + (size_t)c * W;
#pragma unroll
        for (int i = 0; i < V * W; i += V) VecIO<T, V>::load(flat + i, p + i);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = flat[i * W + j];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        bias[i] = !bp ? 0.f
                  : w_f32 ? reinterpret_cast<const float*>(bp)[c + i]
                          : to_f32(reinterpret_cast<const T*>(bp)[c + i]);
}

// Input row r of sequence b (r >= -(W-1); negative rows come from X0).
template <typename T, int V, int W>
__device__ __forceinline__ void load_row(float* f, const T* xb, const T* X0b, long long xt, int D, int r) {
    if (r >= 0) {
        VecIO<T, V>::load(f, xb + r * xt);
    } else if (X0b) {
        VecIO<T, V>::load(f, X0b + (size_t)(r + W - 1) * D);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 0.f;
    }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const T* __restrict__ x, const void* __restrict__ weight,
                                                       const void* __restrict__ bias, const T* X0,
                                                       const int* __restrict__ lengths, T* __restrict__ y, T* X_T,
                                                       long long xb, long long xt, ConvShape s) {
    const unsigned idx = blockIdx.x * 128u + threadIdx.x;
    if (idx >= s.total) return;
    const unsigned r0 = idx / s.nvec;
    const int c = (idx - r0 * s.nvec) * V;
    const int b = r0 / s.nchunk, chunk = r0 - b * s.nchunk;
    const int t0 = chunk * s.tt, t1 = min(s.T, t0 + s.tt);
    const int n = seq_len(lengths, b, s.T);
    const T* xr = x + b * xb + c;
    const T* X0r = X0 ? X0 + (size_t)b * (W - 1) * s.D + c : nullptr;
    T* yr = y + (size_t)b * s.T * s.D + c;

    float w[W][V], bs[V], win[W][V];  // win[j]: row t - W + 1 + j
    load_taps<T, V, W>(w, bs, weight, bias, c, s.w_f32);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int r = t0 - (W - 1) + j;
        if (r < n) load_row<T, V, W>(win[j], xr, X0r, xt, s.D, r);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = 0.f;
    }
    // The first chunk writes the carried rows. X_T may be X0 itself: only this
    // thread reads these channels of X0, and win holds them all by now.
    if (chunk == 0 && X_T) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int r = n - (W - 1) + j;
            float f[V];
            if (r >= 0) VecIO<T, V>::load(f, xr + r * xt);
            else
#pragma unroll
                for (int jj = 0; jj < W - 1; ++jj)
                    if (r + W - 1 == jj)
#pragma unroll
                        for (int i = 0; i < V; ++i) f[i] = win[jj][i];
            VecIO<T, V>::store(X_T + ((size_t)b * (W - 1) + j) * s.D + c, f);
        }
    }
    for (int tb = t0; tb < t1; tb += kConvBatch) {
        float rows[kConvBatch][V];
#pragma unroll
        for (int k = 0; k < kConvBatch; ++k) {
            if (tb + k < min(t1, n)) VecIO<T, V>::load(rows[k], xr + (tb + k) * xt);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) rows[k][i] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < kConvBatch; ++k) {
            const int t = tb + k;
            if (t >= t1) break;
            float out[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                win[W - 1][i] = rows[k][i];
                float p = bs[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                out[i] = t >= n ? 0.f : s.silu ? p * sigmoidf_fast(p) : p;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
            }
            VecIO<T, V>::store(yr + (size_t)t * s.D, out);
        }
    }
}

// One chunk of tokens: dx of its rows (and dX0 in the first chunk), and the
// chunk's partial dw, dbias. dx_s needs dp up to W - 1 tokens on, so the walk
// runs W - 1 tokens past the chunk; those tokens' dw belongs to the next chunk.
template <typename T, typename TG, int V, int W>
__global__ void __launch_bounds__(128) conv_bwd_kernel(
    const T* __restrict__ x, const void* __restrict__ weight, const void* __restrict__ bias,
    const T* __restrict__ X0, const int* __restrict__ lengths, const TG* __restrict__ dy,
    const float* __restrict__ dX_T, float* __restrict__ dx, float* __restrict__ dX0, float* __restrict__ part,
    long long xb, long long xt, long long gb, long long gt, ConvShape s) {
    const unsigned idx = blockIdx.x * 128u + threadIdx.x;
    if (idx >= s.total) return;
    const unsigned r0 = idx / s.nvec;
    const int c = (idx - r0 * s.nvec) * V;
    const int b = r0 / s.nchunk, chunk = r0 - b * s.nchunk;
    const int t0 = chunk * s.tt, t1 = min(s.T, t0 + s.tt);
    const int n = seq_len(lengths, b, s.T);
    const T* xr = x + b * xb + c;
    const TG* gr = dy + b * gb + c;
    const T* X0r = X0 ? X0 + (size_t)b * (W - 1) * s.D + c : nullptr;

    float w[W][V], bs[V], win[W][V], dw[W][V], db[V], acc[W][V];
    load_taps<T, V, W>(w, bs, weight, bias, c, s.w_f32);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = acc[j][i] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int r = t0 - (W - 1) + j;
        if (r < n) load_row<T, V, W>(win[j], xr, X0r, xt, s.D, r);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = 0.f;
    }
    for (int tb = t0; tb < t1 + W - 1; tb += kConvBatch) {
        float rows[kConvBatch][V], grads[kConvBatch][V];
#pragma unroll
        for (int k = 0; k < kConvBatch; ++k) {
            if (tb + k < min(t1 + W - 1, n)) {
                VecIO<T, V>::load(rows[k], xr + (tb + k) * xt);
                VecIO<TG, V>::load(grads[k], gr + (tb + k) * gt);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) rows[k][i] = grads[k][i] = 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kConvBatch; ++k) {
            const int t = tb + k;
            if (t >= t1 + W - 1) break;
            const int e = t - (W - 1);  // the row whose gradient is complete after this token
            float out[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                win[W - 1][i] = rows[k][i];
                float dp = grads[k][i];  // 0 from n on
                if (s.silu) {
                    float p = bs[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                    const float sg = sigmoidf_fast(p);
                    dp = t < n ? dp * (sg * fmaf(p, 1.f - sg, 1.f)) : 0.f;
                }
                if (t < t1) {
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][i] = fmaf(dp, win[j][i], dw[j][i]);
                    db[i] += dp;
                }
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j][i] = fmaf(w[j][i], dp, acc[j][i]);
                out[i] = acc[0][i];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    acc[j][i] = acc[j + 1][i];
                    win[j][i] = win[j + 1][i];
                }
                acc[W - 1][i] = 0.f;
            }
            const bool lead = chunk == 0 && e < 0;  // a carried row
            if (e < t0 && !lead) continue;
            const int tail = e - (n - (W - 1));  // row of X_T that is input row e
            if (dX_T && tail >= 0 && tail < W - 1) {
                float f[V];
                VecIO<float, V>::load(f, dX_T + ((size_t)b * (W - 1) + tail) * s.D + c);
#pragma unroll
                for (int i = 0; i < V; ++i) out[i] += f[i];
            }
            if (!lead) VecIO<float, V>::store(dx + ((size_t)b * s.T + e) * s.D + c, out);
            else if (dX0) VecIO<float, V>::store(dX0 + ((size_t)b * (W - 1) + e + W - 1) * s.D + c, out);
        }
    }
    float* pr = part + (size_t)r0 * (W + 1) * s.D + c;  // partial sums [b, chunk][W + 1][D]
#pragma unroll
    for (int j = 0; j < W; ++j) VecIO<float, V>::store(pr + (size_t)j * s.D, dw[j]);
    VecIO<float, V>::store(pr + (size_t)W * s.D, db);
}

// dweight [D, W] and dbias [D] from `parts` partials of [W + 1][D]: 32 columns
// x 8 slices of the partials per block, slices added in order.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                          float* __restrict__ db, int parts, int D, int W) {
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const long long cols = (long long)(W + 1) * D;
    const long long col = (long long)blockIdx.x * 32 + lane;
    __shared__ float sm[8][32];
    float a = 0.f;
    dependent_wait();
    if (col < cols)
        for (int p = sl; p < parts; p += 8) a += part[(size_t)p * cols + col];
    sm[sl][lane] = a;
    __syncthreads();
    if (sl == 0 && col < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) a += sm[k][lane];
        const int j = (int)(col / D), d = (int)(col - (long long)j * D);
        if (j < W) dw[(size_t)d * W + j] = a;
        else if (db) db[d] = a;
    }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const T* __restrict__ x, const void* __restrict__ weight,
                                                        const void* __restrict__ bias, T* __restrict__ X,
                                                        T* __restrict__ y, long long xb, ConvShape s) {
    dependent_launch();
    const unsigned idx = blockIdx.x * 128u + threadIdx.x;
    if (idx >= s.total) return;
    const int b = idx / s.nvec;
    const int c = (idx - b * s.nvec) * V;
    float w[W][V], bs[V], win[W][V], out[V];
    dependent_wait();
    T* Xr = X + (size_t)b * (W - 1) * s.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) VecIO<T, V>::load(win[j], Xr + (size_t)j * s.D);
    VecIO<T, V>::load(win[W - 1], x + b * xb + c);
    load_taps<T, V, W>(w, bs, weight, bias, c, s.w_f32);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = bs[i];
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
        out[i] = s.silu ? p * sigmoidf_fast(p) : p;
    }
    VecIO<T, V>::store(y + (size_t)b * s.D + c, out);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) VecIO<T, V>::store(Xr + (size_t)j * s.D, win[j + 1]);
}

// Tokens per thread. A chunk of tt tokens loads W - 1 halo rows and writes one
// set of partials, so longer is better until there are too few threads to keep
// the loads in flight; `want` threads fill the card.
static int conv_tokens(long long per_token, int T, int lo, int hi, long long want) {
    int tt = hi;
    while (tt > lo && per_token * ((T + tt - 1) / tt) < want) tt /= 2;
    return tt;
}

static int conv_fwd_tokens(int B, int T, int nvec) {
    return conv_tokens((long long)B * nvec, T, 8, 32, 148 * 2048);
}
static int conv_bwd_tokens(int B, int T, int nvec) {
    return conv_tokens((long long)B * nvec, T, 16, 128, 148 * 1024);
}
static int conv_chunks(int T, int tt) { return T > 0 ? (T + tt - 1) / tt : 1; }

template <typename F> static bool dispatch_taps(int W, F&& f) {
    switch (W) {
        case 2: f(std::integral_constant<int, 2>()); return true;
        case 3: f(std::integral_constant<int, 3>()); return true;
        case 4: f(std::integral_constant<int, 4>()); return true;
        default: return false;
    }
}

}  // namespace gdr

using namespace gdr;

static gdr_status conv_check(const void* weight, const void* bias, int B, int T, int D, int W, int activation,
                             int dtype, int weight_dtype) {
    if (B < 1 || T < 0 || D < 1 || W < 1 || !dtype_ok(dtype) || !dtype_ok(weight_dtype)) return GDR_ERR_INVALID_ARG;
    if (activation != GDR_ACT_NONE && activation != GDR_ACT_SILU) return GDR_ERR_INVALID_ARG;
    if (!weight) return GDR_ERR_INVALID_ARG;
    if (W < 2 || W > 4) return GDR_ERR_UNSUPPORTED;
    if (weight_dtype != dtype && weight_dtype != GDR_FP32) return GDR_ERR_UNSUPPORTED;
    if (!aligned_to(weight, dtype_size(weight_dtype)) || !aligned_to(bias, dtype_size(weight_dtype)))
        return GDR_ERR_MISALIGNED;
    return GDR_OK;
}

// 16-byte rows: the channel count and every stride a multiple of the vector,
// every pointer aligned to it.
static bool conv_vector(int D, int V, size_t e, const void* weight, std::initializer_list<const void*> ptrs,
                        std::initializer_list<long long> strides) {
    if (D % V || !aligned_to(weight, 16)) return false;
    for (const void* p : ptrs)
        if (!aligned_to(p, e * V < 16 ? e * V : 16)) return false;
    for (long long st : strides)
        if (st % V) return false;
    return true;
}

static cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

extern "C" {

gdr_status gdr_conv_fwd(const void* x, const void* weight, const void* bias, const void* X0, const int* lengths,
                        void* y, void* X_T, const long long* strides, int B, int T, int D, int W, int activation,
                        int dtype, int weight_dtype, void* stream) {
    gdr_status ok = conv_check(weight, bias, B, T, D, W, activation, dtype, weight_dtype);
    if (ok != GDR_OK) return ok;
    if (T > 0 && (!x || !y)) return GDR_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype);
    for (const void* p : {x, X0, (const void*)y, (const void*)X_T})
        if (!aligned_to(p, e)) return GDR_ERR_MISALIGNED;
    if (!aligned_to(lengths, 4)) return GDR_ERR_MISALIGNED;
    const long long xb = strides ? strides[0] : (long long)T * D, xt = strides ? strides[1] : D;
    const int V = dtype == GDR_BF16 ? 8 : 4;
    const bool vec = conv_vector(D, V, e, weight, {x, X0, y, X_T}, {xb, xt});
    ConvShape s = {};
    s.T = T; s.D = D; s.nvec = vec ? D / V : D;
    s.tt = conv_fwd_tokens(B, T, s.nvec);
    s.nchunk = conv_chunks(T, s.tt);
    s.silu = activation == GDR_ACT_SILU;
    s.w_f32 = weight_dtype == GDR_FP32;
    const long long total = (long long)B * s.nchunk * s.nvec;
    if (total > (1ll << 31)) return GDR_ERR_UNSUPPORTED;
    s.total = (unsigned)total;
    const unsigned grid = (unsigned)((total + 127) / 128);
    cudaStream_t st = as_stream(stream);
    dispatch_taps(W, [&](auto wc) {
        constexpr int WT = decltype(wc)::value;
#define GDR_CONV_FWD(TT, VV)                                                                              \
    conv_fwd_kernel<TT, VV, WT><<<grid, 128, 0, st>>>((const TT*)x, weight, bias, (const TT*)X0, lengths, \
                                                      (TT*)y, (TT*)X_T, xb, xt, s)
        if (dtype == GDR_BF16) { if (vec) GDR_CONV_FWD(__nv_bfloat16, 8); else GDR_CONV_FWD(__nv_bfloat16, 1); }
        else { if (vec) GDR_CONV_FWD(float, 4); else GDR_CONV_FWD(float, 1); }
#undef GDR_CONV_FWD
    });
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

size_t gdr_conv_bwd_workspace_size(int B, int T, int D, int W) {
    if (B < 1 || T < 0 || D < 1 || W < 2 || W > 4) return 0;
    // the narrow form (one channel per thread) has at most as many chunks
    const int tt = conv_bwd_tokens(B, T, D % 4 ? D : D / 4);
    return round256((size_t)B * conv_chunks(T, tt) * (W + 1) * D * sizeof(float));
}

gdr_status gdr_conv_bwd(const void* x, const void* weight, const void* bias, const void* X0, const int* lengths,
                        const void* dy, const float* dX_T, float* dx, float* dweight, float* dbias, float* dX0,
                        void* workspace, size_t workspace_bytes, const long long* strides, int B, int T, int D,
                        int W, int activation, int dtype, int weight_dtype, int grad_dtype, void* stream) {
    gdr_status ok = conv_check(weight, bias, B, T, D, W, activation, dtype, weight_dtype);
    if (ok != GDR_OK) return ok;
    if (!dtype_ok(grad_dtype)) return GDR_ERR_INVALID_ARG;
    if (grad_dtype != dtype && grad_dtype != GDR_FP32) return GDR_ERR_UNSUPPORTED;
    if (T > 0 && (!x || !dy || !dx)) return GDR_ERR_INVALID_ARG;
    if (!dweight || (dbias != nullptr) != (bias != nullptr) || (dX0 && !X0)) return GDR_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdr_conv_bwd_workspace_size(B, T, D, W)) return GDR_ERR_INVALID_ARG;
    if (!aligned_to(workspace, 256)) return GDR_ERR_MISALIGNED;
    const size_t e = dtype_size(dtype), eg = dtype_size(grad_dtype);
    if (!aligned_to(x, e) || !aligned_to(X0, e) || !aligned_to(dy, eg)) return GDR_ERR_MISALIGNED;
    for (const void* p : {(const void*)lengths, (const void*)dX_T, (const void*)dx, (const void*)dweight,
                          (const void*)dbias, (const void*)dX0})
        if (!aligned_to(p, 4)) return GDR_ERR_MISALIGNED;
    const long long xb = strides ? strides[0] : (long long)T * D, xt = strides ? strides[1] : D;
    const long long gb = strides ? strides[2] : (long long)T * D, gt = strides ? strides[3] : D;
    const bool vec = conv_vector(D, 4, e, weight, {x, X0}, {xb, xt, gb, gt}) && aligned_to(dy, eg * 4) &&
                     aligned_to(dX_T, 16) && aligned_to(dx, 16) && aligned_to(dX0, 16);
    ConvShape s = {};
    s.T = T; s.D = D; s.nvec = vec ? D / 4 : D;
    // chunks of the vector form whichever runs, so that one workspace size holds
    s.tt = conv_bwd_tokens(B, T, D % 4 ? D : D / 4);
    s.nchunk = conv_chunks(T, s.tt);
    s.silu = activation == GDR_ACT_SILU;
    s.w_f32 = weight_dtype == GDR_FP32;
    const long long total = (long long)B * s.nchunk * s.nvec;
    if (total > (1ll << 31)) return GDR_ERR_UNSUPPORTED;
    s.total = (unsigned)total;
    const unsigned grid = (unsigned)((total + 127) / 128);
    cudaStream_t st = as_stream(stream);
    float* part = reinterpret_cast<float*>(workspace);
    dispatch_taps(W, [&](auto wc) {
        constexpr int WT = decltype(wc)::value;
#define GDR_CONV_BWD(TT, TG, VV)                                                                               \
    conv_bwd_kernel<TT, TG, VV, WT><<<grid, 128, 0, st>>>((const TT*)x, weight, bias, (const TT*)X0, lengths, \
                                                          (const TG*)dy, dX_T, dx, dX0, part, xb, xt, gb, gt, s)
        if (dtype == GDR_FP32) { if (vec) GDR_CONV_BWD(float, float, 4); else GDR_CONV_BWD(float, float, 1); }
        else if (grad_dtype == GDR_FP32) {
            if (vec) GDR_CONV_BWD(__nv_bfloat16, float, 4); else GDR_CONV_BWD(__nv_bfloat16, float, 1);
        } else {
            if (vec) GDR_CONV_BWD(__nv_bfloat16, __nv_bfloat16, 4);
            else GDR_CONV_BWD(__nv_bfloat16, __nv_bfloat16, 1);
        }
#undef GDR_CONV_BWD
    });
    if (cudaGetLastError() != cudaSuccess) return GDR_ERR_LAUNCH;
    const long long cols = (long long)(W + 1) * D;
    return launch_dependent(conv_reduce_kernel, (unsigned)((cols + 31) / 32), 256, 0, st, part, dweight, dbias,
                            B * s.nchunk, D, W) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

gdr_status gdr_conv_step(const void* x, const void* weight, const void* bias, void* X, void* y,
                         const long long* strides, int B, int D, int W, int activation, int dtype,
                         int weight_dtype, void* stream) {
    gdr_status ok = conv_check(weight, bias, B, 1, D, W, activation, dtype, weight_dtype);
    if (ok != GDR_OK) return ok;
    if (!x || !X || !y) return GDR_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned_to(x, e) || !aligned_to(X, e) || !aligned_to(y, e)) return GDR_ERR_MISALIGNED;
    const long long xb = strides ? strides[0] : D;
    const int V = dtype == GDR_BF16 ? 8 : 4;
    const bool vec = conv_vector(D, V, e, weight, {x, X, y}, {xb});
    ConvShape s = {};
    s.T = 1; s.D = D; s.nvec = vec ? D / V : D;
    s.silu = activation == GDR_ACT_SILU;
    s.w_f32 = weight_dtype == GDR_FP32;
    const long long total = (long long)B * s.nvec;
    if (total > (1ll << 31)) return GDR_ERR_UNSUPPORTED;
    s.total = (unsigned)total;
    const unsigned grid = (unsigned)((total + 127) / 128);
    cudaStream_t st = as_stream(stream);
    cudaError_t err = cudaErrorInvalidValue;
    dispatch_taps(W, [&](auto wc) {
        constexpr int WT = decltype(wc)::value;
#define GDR_CONV_STEP(TT, VV)                                                                       \
    err = launch_dependent(conv_step_kernel<TT, VV, WT>, grid, 128, 0, st, (const TT*)x, weight,    \
                           bias, (TT*)X, (TT*)y, xb, s)
        if (dtype == GDR_BF16) { if (vec) GDR_CONV_STEP(__nv_bfloat16, 8); else GDR_CONV_STEP(__nv_bfloat16, 1); }
        else { if (vec) GDR_CONV_STEP(float, 4); else GDR_CONV_STEP(float, 1); }
#undef GDR_CONV_STEP
    });
    return err == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

}  // extern "C"
