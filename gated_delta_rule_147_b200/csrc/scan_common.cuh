// Selective state-space scan: geometry, staging and pair arithmetic shared by
// the forward and backward kernels.
//
// Per channel d and state entry n, with dt = softplus(delta + bias) (or
// delta + bias):
//   h_t = exp(dt_t A[d,n]) h_{t-1} + dt_t u_t B_t[n]
//   y_t = sum_n C_t[n] h_t + D[d] u_t,   out_t = y_t z_t sigmoid(z_t)  (or y_t)
// Channel d of group g reads B[g], C[g]; K = D / G channels share a group.
//
// Geometry. A warp holds CPW channels of one (sequence, group) with all their
// states: a lane owns 4 adjacent states of CH channels, NS lanes cover the
// states (4 NS >= N, the rest padded with A = B = C = 0) and 32 / NS lanes the
// channels. A block of kScanWarps warps holds one such channel tile; its warps
// take segments of L tokens in turn. What is serial, the state passed from a
// segment to the next, is one multiply-add per state and segment: a warp first
// works through its segment from a zero state while it waits.
#pragma once

#include "layer_common.cuh"

namespace gdr {

constexpr int kScanWarps = 8;
constexpr int kScanThreads = 32 * kScanWarps;

__device__ __forceinline__ void lds_quad(f2 (&q)[2], const float* p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    q[0] = v.x;
    q[1] = v.y;
}
__device__ __forceinline__ void sts_quad(float* p, const f2 (&q)[2]) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(q[0], q[1]);
}

// CH adjacent floats of shared memory.
template <int CH> __device__ __forceinline__ void lds_run(float (&f)[CH], const float* p) {
    static_assert(CH == 2 || CH == 4, "channels of a lane");
    if constexpr (CH == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[0] = v.x; f[1] = v.y;
    }
}

// ---- arguments ----
struct ScanArgs {
    const void *u, *delta, *Bm, *Cm, *z, *dy;
    const float *A, *D, *bias, *h0;
    const int* lengths;
    void* y;
    float* h_T;
    long long us[2], ds[2], bs[2], cs[2], zs[2], gs[2];  // batch and token strides
    int T, D_, N, G, K, tiles, softplus, state_vec, bc_vec;
    // backward
    const float* dh_T;
    float *du, *ddelta, *dz, *dh0;
    float* ckpt;    // state at every segment's start, lane order
    float* bcpart;  // dB, dC of each channel tile
    float* prm;     // dA, dD, ddelta_bias of each sequence
    int nseg;       // segments of T tokens
};

template <int NS_, int CH_, int L_> struct ScanGeom {
    static constexpr int NS = NS_, CH = CH_, L = L_;
    static constexpr int NP = 4 * NS;          // padded states
    static constexpr int CL = 32 / NS;         // channel lanes
    static constexpr int CPW = CH * CL;        // channels of a warp (and block)
    static constexpr int SE = (L * CPW + 31) / 32;  // staged token-channels per lane
    static constexpr int BE = (L * NP + 31) / 32;   // staged B (or C) values per lane
    static constexpr int QUADS = CH * 32 * 4;  // floats of a warp's state
};

// Block -> (sequence, group, channel tile), tile fastest: blocks that share
// B and C run together.
struct ScanTile {
    int b, g, tile, c0, kleft, n;
    __device__ __forceinline__ ScanTile(const ScanArgs& a, int cpw) {
        const int blk = blockIdx.x;
        tile = blk % a.tiles;
        const int r = blk / a.tiles;
        g = r % a.G;
        b = r / a.G;
        c0 = g * a.K + tile * cpw;
        kleft = min(cpw, a.K - tile * cpw);
        n = seq_len(a.lengths, b, a.T);
    }
};

// One lane's states of the tile's channels, [D, N] (A) or [B, D, N] layout.
template <typename Gm>
__device__ __forceinline__ void load_states(f2 (&s)[Gm::CH][2], const float* p, const ScanTile& tl, int N, int vec,
                                            int cl, int nl, float scale, bool clamp) {
#pragma unroll
    for (int c = 0; c < Gm::CH; ++c) {
        const int ch = cl * Gm::CH + c;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (ch < tl.kleft && nl * 4 < N) {
            const float* q = p + (size_t)(tl.c0 + ch) * N + nl * 4;
            if (vec) VecIO<float, 4>::load(f, q);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (nl * 4 + i < N) f[i] = q[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] *= scale;
            // A = -inf (a state that holds one token) times dt = 0 of a padded
            // token would be NaN; the lowest number gives the same decays
            if (clamp && f[i] < -3.402823466e38f) f[i] = -3.402823466e38f;
        }
        s[c][0] = pack2(f[0], f[1]);
        s[c][1] = pack2(f[2], f[3]);
    }
}
template <typename Gm>
__device__ __forceinline__ void store_states(float* p, const f2 (&s)[Gm::CH][2], const ScanTile& tl, int N, int vec,
                                             int cl, int nl) {
#pragma unroll
    for (int c = 0; c < Gm::CH; ++c) {
        const int ch = cl * Gm::CH + c;
        if (ch >= tl.kleft || nl * 4 >= N) continue;
        float f[4];
        unpack2(s[c][0], f[0], f[1]);
        unpack2(s[c][1], f[2], f[3]);
        float* q = p + (size_t)(tl.c0 + ch) * N + nl * 4;
        if (vec) VecIO<float, 4>::store(q, f);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (nl * 4 + i < N) q[i] = f[i];
    }
}

// A tile's [L tokens][CPW channels] of one input, as the lanes stage it:
// element i of a lane is token (32 i + lane) / CPW, channel (32 i + lane) % CPW.
// Tokens from n on and channels beyond the tile are not read and give 0.
template <typename T, typename Gm>
__device__ __forceinline__ void fetch_rows(T (&r)[Gm::SE], const T* p, long long st, int t0, const ScanTile& tl,
                                           int lane) {
#pragma unroll
    for (int i = 0; i < Gm::SE; ++i) {
        const int e = 32 * i + lane, step = e / Gm::CPW, ch = e % Gm::CPW;
        r[i] = from_f32<T>(0.f);
        if (step < Gm::L && t0 + step < tl.n && ch < tl.kleft) r[i] = p[(t0 + step) * st + ch];
    }
}
template <typename T, typename Gm>
__device__ __forceinline__ void fetch_vecs(T (&r)[Gm::BE], const T* p, long long st, int t0, const ScanTile& tl, int N,
                                           int lane) {
#pragma unroll
    for (int i = 0; i < Gm::BE; ++i) {
        const int e = 32 * i + lane, step = e / Gm::NP, n = e % Gm::NP;
        r[i] = from_f32<T>(0.f);
        if (step < Gm::L && t0 + step < tl.n && n < N) r[i] = p[(t0 + step) * st + n];
    }
}
template <typename T, typename Gm>
__device__ __forceinline__ void stage_vecs(float* s, const T (&r)[Gm::BE], int lane) {
#pragma unroll
    for (int i = 0; i < Gm::BE; ++i) {
        const int e = 32 * i + lane;
        if (e < Gm::L * Gm::NP) s[e] = to_f32(r[i]);
    }
}

// Named barriers 1..kScanWarps hand a warp its incoming state: the producer
// arrives without waiting, the consumer waits. Used once per segment; a
// producer's next arrival follows, through the chain of segments, the
// consumer's last wait, so the barrier never sees two arrivals in a row.
__device__ __forceinline__ void carry_arrive(int warp) {
    __syncwarp();
    __threadfence_block();
    asm volatile("bar.arrive %0, 64;" ::"r"(warp + 1) : "memory");
}
__device__ __forceinline__ void carry_wait(int warp) {
    __syncwarp();
    asm volatile("bar.sync %0, 64;" ::"r"(warp + 1) : "memory");
}

// Sums V values of each lane over the 2^k lanes whose numbers differ in the
// bits STRIDE .. STRIDE * LANES / 2. While V is even a step halves the values
// a lane keeps (one shuffle per value kept); the lane's bit of that step says
// which half it holds. Returns the number of values left.
template <int V, int LANES, int STRIDE> struct LaneSum {
    static constexpr int left() {
        if constexpr (LANES > 1 && V % 2 == 0) return LaneSum<V / 2, LANES / 2, STRIDE * 2>::left();
        else return V;
    }
    template <int VV> static __device__ __forceinline__ void run(float (&v)[VV], int lane) {
        if constexpr (LANES > 1 && V % 2 == 0) {
            const bool up = lane & STRIDE;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float keep = up ? v[V / 2 + i] : v[i], give = up ? v[i] : v[V / 2 + i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, STRIDE);
            }
            LaneSum<V / 2, LANES / 2, STRIDE * 2>::run(v, lane);
        } else if constexpr (LANES > 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], STRIDE);
            LaneSum<V, LANES / 2, STRIDE * 2>::run(v, lane);
        }
    }
    // index of value 0 held by this lane among the original V, and whether it
    // is the one lane of its copies that writes
    static __device__ __forceinline__ int first(int lane) {
        if constexpr (LANES > 1 && V % 2 == 0)
            return ((lane & STRIDE) ? V / 2 : 0) + LaneSum<V / 2, LANES / 2, STRIDE * 2>::first(lane);
        else if constexpr (LANES > 1) return LaneSum<V, LANES / 2, STRIDE * 2>::first(lane);
        else return 0;
    }
    static __device__ __forceinline__ bool owner(int lane) {
        if constexpr (LANES > 1 && V % 2 == 0) return LaneSum<V / 2, LANES / 2, STRIDE * 2>::owner(lane);
        else if constexpr (LANES > 1) return !(lane & STRIDE) && LaneSum<V, LANES / 2, STRIDE * 2>::owner(lane);
        else return true;
    }
};

// Lanes that share a channel's states, by the state size.
inline int scan_lanes(int N) {
    int ns = 1;
    while (4 * ns < N) ns *= 2;
    return ns;
}

}  // namespace gdr
