// Short causal depthwise convolution: forward, backward and single token.
//
// Per channel, with W taps and the W - 1 inputs before the sequence carried
// in X0 (zeros without it):
//   p_t = bias + sum_j w_j x_{t-W+1+j},   y_t = p_t sigmoid(p_t)  (or p_t),
//   X_T = the last W - 1 inputs.
// Backward, with dp_t = dy_t dy/dp (sigmoid(p)(1 + p(1 - sigmoid(p)))):
//   dx_s = sum_j w_j dp_{s+W-1-j},  dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t.
//
// Bound by HBM: a token-channel is read once and written once. The kernels come
// near that only with few instructions per element (first version: 23 forward,
// 50 backward, the issue slots 73% and 68% busy), so: a thread owns V adjacent
// channels as packed pairs of fp32, walks `tt` tokens with the last W - 1 inputs
// in registers (a row is loaded once per chunk, plus W - 1 halo rows that L2
// serves), and tokens whose batch lies inside chunk and sequence take a path
// without conditions. The rows of the next batch are on their way meanwhile.
// Threads are numbered with the channel vector fastest, so narrow layers fill
// warps too. All sums are fp32; y is rounded once, gradients are fp32.
#include "layer_common.cuh"

namespace gdr {

// Channels of a thread and tokens of a batch. Forward, 2 x 4096 x 8192 bf16, 4
// taps: 4 channels and 4 tokens 56.6 us (4.7 TB/s), 4 and 8 63.8, 8 and 4 60.7.
// Backward, 4 x 4096 x 6144: 4 and 4 164 us (4.9 TB/s), 4 and 2 about 190, 2 and 4
// about 200.
constexpr int kConvVec = 4, kConvAhead = 4;
// Backward: a chunk's dweight and dbias are kConvSums sums of 32 tokens or more, 64
// at most, each left in shared memory when it is complete. One sum over a chunk of
// 228 tokens (the case above) had twice the error of torch's sums in fp32, 2.9e-7;
// these have 1.7e-7 (torch's 1.4e-7), in the same time. Chunks of 64 tokens take 195 us.
constexpr int kConvSums = 4;

struct ConvShape {
    int T, D, nvec, nchunk, tt, silu, w_f32;
    int sub, subs;   // backward: tokens of a sum, sums of a chunk
    unsigned total;  // threads: B * nchunk * nvec
};

// Filter taps and bias of V channels (`left` of them real).
template <typename T, int V, int W, int HOW>
__device__ __forceinline__ void load_taps(f2 (&w)[W][V / 2], f2 (&bias)[V / 2], const void* weight, const void* bp,
                                          int c, int left, int w_f32) {
    float flat[V * W], bf[V];  // [V][W], as the rows of [D, W] lie
    if (HOW == kWholeRow && w_f32) {
#pragma unroll
        for (int i = 0; i < V * W; i += 4)
            VecIO<float, 4>::load(flat + i, reinterpret_cast<const float*>(weight) + (size_t)c * W + i);
    } else if (HOW == kWholeRow) {
#pragma unroll
        for (int i = 0; i < V * W; i += V)
            VecIO<T, V>::load(flat + i, reinterpret_cast<const T*>(weight) + (size_t)c * W + i);
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i)
            flat[i] = i / W >= left ? 0.f
                      : w_f32 ? reinterpret_cast<const float*>(weight)[(size_t)c * W + i]
                              : to_f32(reinterpret_cast<const T*>(weight)[(size_t)c * W + i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        bf[i] = !bp || i >= left ? 0.f
                : w_f32 ? reinterpret_cast<const float*>(bp)[c + i]
                        : to_f32(reinterpret_cast<const T*>(bp)[c + i]);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        bias[i] = pack2(bf[2 * i], bf[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = pack2(flat[2 * i * W + j], flat[(2 * i + 1) * W + j]);
    }
}

// The W - 1 inputs before row t0 of a sequence of n tokens (negative rows come
// from X0); rows from n on are not read.
template <typename T, int V, int W, int HOW>
__device__ __forceinline__ void load_window(f2 (&win)[W][V / 2], const T* xr, const T* X0r, long long xt, int D, int t0,
                                            int n, int left) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int r = t0 - (W - 1) + j;
        RowIO<T, V, HOW> row;
        row.zero();
        if (r >= 0 && r < n) row.load(xr + r * xt, left);
        else if (r < 0 && X0r) row.load(X0r + (size_t)(r + W - 1) * D, left);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) win[j][i] = row.pair(i);
    }
}

template <int P, int W> __device__ __forceinline__ void slide(f2 (&win)[W][P]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i];
}

template <typename T, int V, int W, int HOW>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const T* __restrict__ x, const void* __restrict__ weight,
                                                       const void* __restrict__ bias, const T* X0,
                                                       const int* __restrict__ lengths, T* __restrict__ y, T* X_T,
                                                       long long xb, long long xt, ConvShape s) {
    constexpr int P = V / 2, K = kConvAhead;
    using Row = RowIO<T, V, HOW>;
    const unsigned idx = blockIdx.x * 128u + threadIdx.x;
    if (idx >= s.total) return;
    const unsigned r0 = idx / s.nvec;
    const int c = (idx - r0 * s.nvec) * V, left = s.D - c;
    const int b = r0 / s.nchunk, chunk = r0 - b * s.nchunk;
    const int t0 = chunk * s.tt, t1 = min(s.T, t0 + s.tt);
    const int n = seq_len(lengths, b, s.T);
    const T* xr = x + b * xb + c;
    const T* X0r = X0 ? X0 + (size_t)b * (W - 1) * s.D + c : nullptr;
    T* yr = y + ((size_t)b * s.T + t0) * s.D + c;

    f2 w[W][P], bs[P], win[W][P];  // win[j]: row t - W + 1 + j
    load_taps<T, V, W, HOW>(w, bs, weight, bias, c, left, s.w_f32);
    load_window<T, V, W, HOW>(win, xr, X0r, xt, s.D, t0, n, left);
    // The first chunk writes the carried rows. X_T may be X0 itself: only this
    // thread reads these channels of X0, and win holds them all by now.
    if (chunk == 0 && X_T) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int r = n - (W - 1) + j;
            f2 f[P];
            if (r >= 0) {
                Row row;
                row.load(xr + r * xt, left);
#pragma unroll
                for (int i = 0; i < P; ++i) f[i] = row.pair(i);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) f[i] = win[0][i];
#pragma unroll
                for (int jj = 1; jj < W - 1; ++jj)
                    if (r + W - 1 == jj)
#pragma unroll
                        for (int i = 0; i < P; ++i) f[i] = win[jj][i];
            }
            Row::store(X_T + ((size_t)b * (W - 1) + j) * s.D + c, f, left);
        }
    }
    const int end = min(t1, n);
    Row next[K];
    const T* xp = xr + t0 * xt;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        next[k].zero();
        if (t0 + k < end) next[k].load(xp + k * xt, left);
    }
    for (int tb = t0; tb < t1; tb += K) {
        Row rows[K];
        xp += K * xt;
#pragma unroll
        for (int k = 0; k < K; ++k) rows[k] = next[k];
        if (tb + 2 * K <= end) {
#pragma unroll
            for (int k = 0; k < K; ++k) next[k].load(xp + k * xt, left);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tb + K + k < end) next[k].load(xp + k * xt, left);
        }
        const bool whole = tb + K <= end;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f2 out[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                win[W - 1][i] = rows[k].pair(i);
                out[i] = bs[i];
#pragma unroll
                for (int j = 0; j < W; ++j) out[i] = fma2(w[j][i], win[j][i], out[i]);
            }
            if (s.silu) {
#pragma unroll
                for (int i = 0; i < P; ++i) out[i] = mul2(out[i], sigmoid2(out[i]));
            }
            slide(win);
            if (!whole && tb + k >= n) {
#pragma unroll
                for (int i = 0; i < P; ++i) out[i] = both2(0.f);
            }
            if (whole || tb + k < t1) Row::store(yr, out, left);
            yr += s.D;
        }
    }
}

// Blocks per SM of the backward kernel, by the bytes of an element of x and of dy:
// two where three would spill. Without the bound the compiler places the loads of
// the case above so that it takes 209 us.
constexpr int conv_bwd_blocks(int bytes, int W, int how) { return bytes == 8 && W == 4 && how != kWholeRow ? 2 : 3; }

// One chunk of tokens: dx of its rows (and dX0 in the first chunk), and the
// chunk's partial dw, dbias. dx_s needs dp up to W - 1 tokens on, so the walk
// runs W - 1 tokens past the chunk; those tokens' dw belongs to the next chunk.
template <typename T, typename TG, int V, int W, int HOW>
__global__ void __launch_bounds__(128, conv_bwd_blocks(sizeof(T) + sizeof(TG), W, HOW)) conv_bwd_kernel(
    const T* __restrict__ x, const void* __restrict__ weight, const void* __restrict__ bias,
    const T* __restrict__ X0, const int* __restrict__ lengths, const TG* __restrict__ dy,
    const float* __restrict__ dX_T, float* __restrict__ dx, float* __restrict__ dX0, float* __restrict__ part,
    long long xb, long long xt, long long gb, long long gt, ConvShape s) {
    constexpr int P = V / 2, K = kConvAhead;
    using Row = RowIO<T, V, HOW>;
    using Grad = RowIO<TG, V, HOW>;
    using Out = RowIO<float, V, HOW>;
    const unsigned idx = blockIdx.x * 128u + threadIdx.x;
    if (idx >= s.total) return;
    const unsigned r0 = idx / s.nvec;
    const int c = (idx - r0 * s.nvec) * V, left = s.D - c;
    const int b = r0 / s.nchunk, chunk = r0 - b * s.nchunk;
    const int t0 = chunk * s.tt, t1 = min(s.T, t0 + s.tt), stop = t1 + W - 1;
    const int n = seq_len(lengths, b, s.T);
    const T* xr = x + b * xb + c;
    const T* X0r = X0 ? X0 + (size_t)b * (W - 1) * s.D + c : nullptr;

    f2 w[W][P], bs[P], win[W][P], dw[W][P], db[P], acc[W][P];  // acc[j]: dx of row t - W + 1 + j so far
    load_taps<T, V, W, HOW>(w, bs, weight, bias, c, left, s.w_f32);
    load_window<T, V, W, HOW>(win, xr, X0r, xt, s.D, t0, n, left);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j][i] = both2(0.f);
    // one token: dp from its row and gradient, its share of the sums (SUM), and
    // the gradient of row t - W + 1, complete after it
    auto token = [&](const Row& row, const Grad& grad, bool sum, f2 (&out)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            win[W - 1][i] = row.pair(i);
            f2 dp = grad.pair(i);
            if (s.silu) {
                f2 p = bs[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fma2(w[j][i], win[j][i], p);
                const f2 sg = sigmoid2(p);
                // sg (1 + p (1 - sg))
                dp = mul2(dp, mul2(sg, fma2(p, fma2(sg, both2(-1.f), both2(1.f)), both2(1.f))));
            }
            if (sum) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][i] = fma2(dp, win[j][i], dw[j][i]);
                db[i] = add2(db[i], dp);
            }
            out[i] = fma2(w[0][i], dp, acc[0][i]);
#pragma unroll
            for (int j = 1; j < W; ++j) acc[j - 1][i] = j < W - 1 ? fma2(w[j][i], dp, acc[j][i]) : mul2(w[j][i], dp);
        }
        slide(win);
    };
    const int end = min(stop, n);  // tokens from here on are not read
    Row xnext[K];
    Grad gnext[K];
    const T* xp = xr + t0 * xt;
    const TG* gp = dy + b * gb + c + t0 * gt;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        xnext[k].zero();
        gnext[k].zero();
        if (t0 + k < end) {
            xnext[k].load(xp + k * xt, left);
            gnext[k].load(gp + k * gt, left);
        }
    }
    float* dxr = dx + ((long long)b * s.T + t0 - (W - 1)) * s.D + c;  // row t - W + 1
    static_assert(V == 4, "sums in quads");
    __shared__ __align__(16) float sums[kConvSums][W + 1][128][V];  // a thread's own
#pragma unroll 1
    for (int q = 0, tg = t0; q < s.subs; ++q, tg += s.sub) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            db[i] = both2(0.f);
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][i] = both2(0.f);
        }
        const int te = q + 1 == s.subs ? stop : min(stop, tg + s.sub);
        for (int tb = tg; tb < te; tb += K) {
            Row rows[K];
            Grad grads[K];
            xp += K * xt;
            gp += K * gt;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                rows[k] = xnext[k];
                grads[k] = gnext[k];
            }
            if (tb + 2 * K <= end) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    xnext[k].load(xp + k * xt, left);
                    gnext[k].load(gp + k * gt, left);
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    xnext[k].zero();
                    gnext[k].zero();
                    if (tb + K + k < end) {
                        xnext[k].load(xp + k * xt, left);
                        gnext[k].load(gp + k * gt, left);
                    }
                }
            }
            if (tb >= t0 + W - 1 && tb + K <= min(t1, n)) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    f2 out[P];
                    token(rows[k], grads[k], true, out);
                    Out::store(dxr, out, left);
                    dxr += s.D;
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < K; ++k) {
                    const int t = tb + k, e = t - (W - 1);
                    Row row = rows[0];  // rows[k] without an index that is not constant
                    Grad grad = grads[0];
#pragma unroll
                    for (int q = 1; q < K; ++q)
                        if (q == k) { row = rows[q]; grad = grads[q]; }
                    f2 out[P];
                    // a token that is not read only moves the running gradients on
                    if (t >= n) {
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            out[i] = acc[0][i];
#pragma unroll
                            for (int j = 1; j < W; ++j) acc[j - 1][i] = j < W - 1 ? acc[j][i] : both2(0.f);
                        }
                        slide(win);
                    } else {
                        token(row, grad, t < t1, out);
                    }
                    const bool lead = chunk == 0 && e < 0;  // a carried row
                    const int tail = e - (n - (W - 1));     // row of X_T that is input row e
                    if (t < stop && (e >= t0 || lead)) {
                        if (dX_T && tail >= 0 && tail < W - 1) {
                            Out d;
                            d.load(dX_T + ((size_t)b * (W - 1) + tail) * s.D + c, left);
#pragma unroll
                            for (int i = 0; i < P; ++i) out[i] = add2(out[i], d.pair(i));
                        }
                        if (!lead) Out::store(dxr, out, left);
                        else if (dX0) Out::store(dX0 + ((size_t)b * (W - 1) + e + W - 1) * s.D + c, out, left);
                    }
                    dxr += s.D;
                }
            }
        }
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            const f2 (&r)[P] = j < W ? dw[j < W ? j : 0] : db;
            *reinterpret_cast<ulonglong2*>(sums[q][j][threadIdx.x]) = make_ulonglong2(r[0], r[1]);
        }
    }
    float* pr = part + (size_t)r0 * (W + 1) * s.D + c;  // partial sums [b, chunk][W + 1][D]
#pragma unroll 1
    for (int j = 0; j <= W; ++j) {
        f2 f[P] = {both2(0.f), both2(0.f)};
        for (int q = 0; q < s.subs; ++q) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sums[q][j][threadIdx.x]);
            f[0] = add2(f[0], v.x);
            f[1] = add2(f[1], v.y);
        }
        Out::store(pr + (size_t)j * s.D, f, left);
    }
}

// dweight [D, W] and dbias [D] from `parts` partials of [W + 1][D]: 32 columns
// x 8 slices of the partials per block, slices added in order. Sums of 16 partials
// are added in 64 bits: a narrow layer has thousands of partials (8 x 16384 tokens x
// 64 channels: 8192). All 16 loads are on their way together, those beyond the
// last partial repeat it.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                          float* __restrict__ db, int parts, int D, int W) {
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const long long cols = (long long)(W + 1) * D;
    const long long col = (long long)blockIdx.x * 32 + lane;
    __shared__ double sm[8][32];
    double a = 0.;
    dependent_wait();
    if (col < cols)
        for (int p0 = sl; p0 < parts; p0 += 8 * 16) {
            float v[16], t = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = part[(size_t)min(p0 + 8 * k, parts - 1) * cols + col];
#pragma unroll
            for (int k = 0; k < 16; ++k) t += p0 + 8 * k < parts ? v[k] : 0.f;
            a += t;
        }
    sm[sl][lane] = a;
    __syncthreads();
    if (sl == 0 && col < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) a += sm[k][lane];
        const int j = (int)(col / D), d = (int)(col - (long long)j * D);
        if (j < W) dw[(size_t)d * W + j] = (float)a;
        else if (db) db[d] = (float)a;
    }
}

// SEQ sequences of V channels per thread: with several, the taps are read once
// for all of them and more rows are on their way.
template <typename T, int V, int W, int HOW, int SEQ>
__global__ void __launch_bounds__(128) conv_step_kernel(const T* __restrict__ x, const void* __restrict__ weight,
                                                        const void* __restrict__ bias, T* __restrict__ X,
                                                        T* __restrict__ y, long long xb, int B, ConvShape s) {
    constexpr int P = V / 2;
    using Row = RowIO<T, V, HOW>;
    dependent_launch();
    const unsigned idx = blockIdx.x * 128u + threadIdx.x;
    if (idx >= s.total) return;
    const int b0 = idx / s.nvec;
    const int c = (idx - b0 * s.nvec) * V, left = s.D - c;
    f2 w[W][P], bs[P];
    Row rows[SEQ][W];
    dependent_wait();
#pragma unroll
    for (int q = 0; q < SEQ; ++q) {
        const int b = b0 * SEQ + q;
        if (b >= B) continue;
        const T* Xr = X + (size_t)b * (W - 1) * s.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) rows[q][j].load(Xr + (size_t)j * s.D, left);
        rows[q][W - 1].load(x + b * xb + c, left);
    }
    load_taps<T, V, W, HOW>(w, bs, weight, bias, c, left, s.w_f32);
#pragma unroll
    for (int q = 0; q < SEQ; ++q) {
        const int b = b0 * SEQ + q;
        if (b >= B) continue;
        f2 out[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            out[i] = bs[i];
#pragma unroll
            for (int j = 0; j < W; ++j) out[i] = fma2(w[j][i], rows[q][j].pair(i), out[i]);
            if (s.silu) out[i] = mul2(out[i], sigmoid2(out[i]));
        }
        Row::store(y + (size_t)b * s.D + c, out, left);
        T* Xr = X + (size_t)b * (W - 1) * s.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            f2 f[P];
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = rows[q][j + 1].pair(i);
            Row::store(Xr + (size_t)j * s.D, f, left);
        }
    }
}

// Tokens per thread. A chunk of tt tokens loads W - 1 halo rows and writes one
// set of partials, so longer is better, up to `hi`; but the threads should come
// to a whole number of waves of `wave` threads (two here), and to enough of them
// that the loads stay in flight. Backward of the case above: 256 tokens make 1.7
// waves and take 171 us.
static int conv_tokens(long long per_token, int T, int lo, int hi, long long wave) {
    const long long chunks = 2 * wave / per_token;
    long long tt = chunks > 0 ? (T + chunks - 1) / chunks : hi;
    tt = (tt + kConvAhead - 1) / kConvAhead * kConvAhead;
    return (int)(tt < lo ? lo : tt > hi ? hi : tt);
}
// Resident threads: 7 blocks of 128 (70 registers) and 3 (160) to an SM.
static int conv_fwd_tokens(int B, int T, int nvec) { return conv_tokens((long long)B * nvec, T, 8, 64, 148 * 7 * 128); }
static int conv_bwd_tokens(int B, int T, int nvec) { return conv_tokens((long long)B * nvec, T, 16, 256, 148 * 3 * 128); }
// Tokens of one sum in a chunk of tt, whole batches.
static int conv_sum_tokens(int tt) {
    const int sub = (tt + kConvSums - 1) / kConvSums;
    return sub < 32 ? 32 : (sub + kConvAhead - 1) / kConvAhead * kConvAhead;
}
static int conv_vectors(int D) { return (D + kConvVec - 1) / kConvVec; }
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
    if (W < 2 || W > 4 || !axes_fit({B, T, D})) return GDR_ERR_UNSUPPORTED;
    if (weight_dtype != dtype && weight_dtype != GDR_FP32) return GDR_ERR_UNSUPPORTED;
    if (!aligned_to(weight, dtype_size(weight_dtype)) || !aligned_to(bias, dtype_size(weight_dtype)))
        return GDR_ERR_MISALIGNED;
    return GDR_OK;
}

// How rows are accessed: vectors or pairs where the channel count and every
// stride are multiples of theirs and every pointer is aligned to them.
struct RowPtr { const void* p; size_t e; };
static int conv_access(int D, const void* weight, std::initializer_list<RowPtr> ptrs,
                       std::initializer_list<long long> strides) {
    auto fits = [&](int m) {
        bool ok = D % m == 0;
        for (const RowPtr& r : ptrs) ok = ok && aligned_to(r.p, r.e * m);
        for (long long st : strides) ok = ok && st % m == 0;
        return ok;
    };
    return fits(kConvVec) && aligned_to(weight, 16) ? kWholeRow : fits(2) ? kPairRow : kSingleRow;
}
template <typename F> static void dispatch_access(int how, F&& f) {
    if (how == kWholeRow) f(std::integral_constant<int, kWholeRow>());
    else if (how == kPairRow) f(std::integral_constant<int, kPairRow>());
    else f(std::integral_constant<int, kSingleRow>());
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
    const int how = conv_access(D, weight, {{x, e}, {X0, e}, {y, e}, {X_T, e}}, {xb, xt});
    ConvShape s = {};
    s.T = T; s.D = D; s.nvec = conv_vectors(D);
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
        dispatch_access(how, [&](auto hc) {
            constexpr int WT = decltype(wc)::value, HOW = decltype(hc)::value;
#define GDR_CONV_FWD(TT)                                                                                             \
    conv_fwd_kernel<TT, kConvVec, WT, HOW><<<grid, 128, 0, st>>>((const TT*)x, weight, bias, (const TT*)X0, lengths, \
                                                                 (TT*)y, (TT*)X_T, xb, xt, s)
            if (dtype == GDR_BF16) GDR_CONV_FWD(__nv_bfloat16);
            else GDR_CONV_FWD(float);
#undef GDR_CONV_FWD
        });
    });
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

size_t gdr_conv_bwd_workspace_size(int B, int T, int D, int W) {
    if (B < 1 || T < 0 || D < 1 || W < 2 || W > 4 || !axes_fit({B, T, D})) return 0;
    const int tt = conv_bwd_tokens(B, T, conv_vectors(D));
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
    const int how = conv_access(D, weight, {{x, e}, {X0, e}, {dy, eg}, {dX_T, 4}, {dx, 4}, {dX0, 4}}, {xb, xt, gb, gt});
    ConvShape s = {};
    s.T = T; s.D = D; s.nvec = conv_vectors(D);
    s.tt = conv_bwd_tokens(B, T, s.nvec);
    s.sub = conv_sum_tokens(s.tt);
    s.subs = (s.tt + s.sub - 1) / s.sub;
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
        dispatch_access(how, [&](auto hc) {
            constexpr int WT = decltype(wc)::value, HOW = decltype(hc)::value;
#define GDR_CONV_BWD(TT, TG)                                                                                         \
    conv_bwd_kernel<TT, TG, kConvVec, WT, HOW><<<grid, 128, 0, st>>>((const TT*)x, weight, bias, (const TT*)X0,      \
                                                                     lengths, (const TG*)dy, dX_T, dx, dX0, part, xb, \
                                                                     xt, gb, gt, s)
            if (dtype == GDR_FP32) GDR_CONV_BWD(float, float);
            else if (grad_dtype == GDR_FP32) GDR_CONV_BWD(__nv_bfloat16, float);
            else GDR_CONV_BWD(__nv_bfloat16, __nv_bfloat16);
#undef GDR_CONV_BWD
        });
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
    const int how = conv_access(D, weight, {{x, e}, {X, e}, {y, e}}, {xb});
    ConvShape s = {};
    s.T = 1; s.D = D; s.nvec = conv_vectors(D);
    s.silu = activation == GDR_ACT_SILU;
    s.w_f32 = weight_dtype == GDR_FP32;
    // four sequences a thread where that leaves 148 x 1024 threads, 1.1 waves of the
    // 7 blocks of 128 (72 registers) that an SM holds: 12288 channels in bf16, 64
    // sequences 4.0 us with one a thread and 5.1 with four, 200 8.9 both, 256 10.5 and
    // 10.3, 512 18.9 and 17.8
    const bool several = (long long)B * s.nvec >= 4ll * 148 * 1024;
    const long long total = (long long)(several ? (B + 3) / 4 : B) * s.nvec;
    if (total > (1ll << 31)) return GDR_ERR_UNSUPPORTED;
    s.total = (unsigned)total;
    const unsigned grid = (unsigned)((total + 127) / 128);
    cudaStream_t st = as_stream(stream);
    cudaError_t err = cudaErrorInvalidValue;
    dispatch_taps(W, [&](auto wc) {
        dispatch_access(how, [&](auto hc) {
            constexpr int WT = decltype(wc)::value, HOW = decltype(hc)::value;
#define GDR_CONV_STEP(TT, SEQ)                                                                                       \
    err = launch_dependent(conv_step_kernel<TT, kConvVec, WT, HOW, SEQ>, grid, 128, 0, st, (const TT*)x, weight, bias, \
                           (TT*)X, (TT*)y, xb, B, s)
            if (dtype == GDR_BF16) {
                if (several) GDR_CONV_STEP(__nv_bfloat16, 4); else GDR_CONV_STEP(__nv_bfloat16, 1);
            } else {
                if (several) GDR_CONV_STEP(float, 4); else GDR_CONV_STEP(float, 1);
            }
#undef GDR_CONV_STEP
        });
    });
    return err == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

}  // extern "C"
