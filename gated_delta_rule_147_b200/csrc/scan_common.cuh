// Selective state-space scan: geometry, staging and exchange shared by the
// forward and backward kernels.
//
// Per channel d and state entry n, with dt = softplus(delta + bias) (or
// delta + bias):
//   h_t = exp(dt_t A[d,n]) h_{t-1} + dt_t u_t B_t[n]
//   y_t = sum_n C_t[n] h_t + D[d] u_t,   out_t = y_t z_t sigmoid(z_t)  (or y_t)
// Channel d of group g reads B[g], C[g]; K = D / G channels share a group.
//
// Geometry. Two kinds of warps share a block, one of each on every scheduler.
// Four walkers hold a tile of CPW channels each with all their states: a lane
// owns 4 adjacent states of 2 channels, NS lanes cover the states (4 NS >= N,
// the rest padded with A = B = C = 0) and 32 / NS lanes the channels. Four
// helpers turn the inputs of the block's CB = 4 CPW channels into what a walker
// reads per token (dt, dt u; B and C once for the block), LT tokens ahead of
// them, and its sums into outputs, LT tokens behind; one barrier per LT tokens.
// So a walker's stream is the recurrence alone, and the softplus, gates,
// conversions and global accesses fill the issue slots between its exponentials.
// (All of it in one warp, with segments of 8 tokens per warp and their states
// joined by a barrier per 64 tokens, ran at 0.47 instructions per cycle: 856 us
// for 4 x 4096 tokens x 4096 channels x 16 states, against 490 us.)
#pragma once

#include "layer_common.cuh"

namespace gdr {

constexpr int kWalkers = 4, kHelperThreads = 128, kScanThreads = 32 * kWalkers + kHelperThreads;

__device__ __forceinline__ void lds_quad(f2 (&q)[2], const float* p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    q[0] = v.x;
    q[1] = v.y;
}
__device__ __forceinline__ void sts_quad(float* p, const f2 (&q)[2]) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(q[0], q[1]);
}

// ---- arguments ----
struct ScanArgs {
    const void *u, *delta, *Bm, *Cm, *z, *dy;
    const float *A, *D, *bias, *h0;
    const int* lengths;
    void* y;
    float* h_T;
    long long us[2], ds[2], bs[2], cs[2], zs[2], gs[2];  // batch and token strides
    int T, D_, N, G, K, tiles, softplus;
    int state_vec, out_vec;  // 16-byte state accesses, wide stores of output rows
    int bc_vec, act_vec;     // alignment of B and C, and of the token rows (kSingle, kWhole, kPairs)
    // backward
    const float* dh_T;
    float *du, *ddelta, *dz, *dh0;
    float* ckpt;    // state every Seg tokens, lane order
    float* bcpart;  // dB, dC of each block's channels
    float* prm;     // dA, dD, ddelta_bias of each sequence and chunk
    int segs;       // segments of T tokens
    // time split: chunks of `chunk` tokens, `chunks` of them; maps of each (decay, end)
    int chunk, chunks;
    float *ends, *grad_ends;
};

template <int NS_, int CH_, int VW_, int STEPS_> struct ScanGeom {
    static constexpr int NS = NS_, CH = CH_;
    static constexpr int NP = 4 * NS;               // padded states
    static constexpr int CL = 32 / NS;              // channel lanes
    static constexpr int CPW = CH * CL;             // channels of a walker
    static constexpr int CB = kWalkers * CPW;       // channels of a block
    static constexpr int NQ = NS < 4 ? NS : 4;      // partial sums over the states that go to shared memory
    static constexpr int QUADS = CH * 32 * 4;       // floats of a walker's state
    static constexpr int LT = STEPS_ * (NS * 4 >= 8 * CH ? 16 : NS * 4 >= 4 * CH ? 8 : 4);  // tokens of a step: bounded by shared memory
    static constexpr int Seg = NS <= 2 ? 4 : 8;     // tokens of a backward segment, likewise
    // the helpers move rows in vectors of VW channels
    static constexpr int VW = VW_ < CB ? VW_ : CB, VPT = CB / VW;
};
// Forward, 4 x 4096 tokens x 4096 channels x 16 states (490 us): 2 channels a lane
// and 2 blocks per SM; 1 channel and 4 blocks took 1.21 times as long, 1 and 3
// 1.29 times. Backward, its checkpoints too, 2 x 4096 x 4096 x 16, ragged (1030
// us): 1 channel and 2 blocks; 2 and 1 took 1.17 times as long. The vectors give
// every helper thread work with 16 states.
constexpr int kFwdBlocks = 2, kBwdBlocks = 2;
// Steps of 16 tokens with 16 states (8 took 1.08 times as long), of 32 where no
// sums are kept.
template <int NS> using ScanFwdGeom = ScanGeom<NS, 2, 4, 1>;
template <int NS> using ScanEndsGeom = ScanGeom<NS, 2, 4, 2>;
template <int NS> using ScanBwdGeom = ScanGeom<NS, 1, 2, 1>;
template <int NS> using ScanCkptGeom = ScanGeom<NS, 1, 2, 2>;
constexpr int scan_segment(int ns) { return ns <= 2 ? 4 : 8; }

// Block -> (sequence, group, channel tile, chunk of tokens), tile fastest:
// blocks that share B and C run together. Tokens [t0, n) are this chunk's,
// rows [t0, t1) its outputs'.
struct ScanTile {
    int b, g, tile, part, c0, kleft, t0, t1, n;
    size_t unit;  // of (sequence, group, tile)
    __device__ __forceinline__ ScanTile(const ScanArgs& a, int cb) {
        unsigned blk = blockIdx.x;
        tile = blk % (unsigned)a.tiles;
        blk /= (unsigned)a.tiles;
        part = blk % (unsigned)a.chunks;
        blk /= (unsigned)a.chunks;
        g = blk % (unsigned)a.G;
        b = blk / (unsigned)a.G;
        unit = ((size_t)b * a.G + g) * a.tiles + tile;
        c0 = g * a.K + tile * cb;
        kleft = min(cb, a.K - tile * cb);
        t0 = part * a.chunk;
        t1 = a.T - t0 < a.chunk ? a.T : t0 + a.chunk;
        n = max(t0, min(t1, seq_len(a.lengths, b, a.T)));
    }
};

// Place of a block's channel among the values of one token in shared memory:
// element j of the helpers' vector k at j VPT + k, so that helpers (one j at a
// time) and walkers (CL adjacent places) both go through the banks in order. With
// channels in their own order helpers met 4-way conflicts, and the kernel took
// 1.5 times as long. Walker w holds the places from w CPW on.
template <typename Gm> __device__ __forceinline__ int channel_place(int ch) { return ch % Gm::VW * Gm::VPT + ch / Gm::VW; }
template <typename Gm> __device__ __forceinline__ int place_channel(int place) {
    return place % Gm::VPT * Gm::VW + place / Gm::VPT;
}
template <typename Gm> __device__ __forceinline__ int lane_place(int walker, int c, int cl) {
    return (walker * Gm::CH + c) * Gm::CL + cl;
}

// One lane's states of its channels (places p0, p0 + CL, ..), [D, N] (A, as decay
// rates with RATE) or [B, D, N] layout.
template <typename Gm, bool RATE>
__device__ __forceinline__ void load_states(f2 (&s)[Gm::CH][2], const float* p, const ScanTile& tl, int N, int vec,
                                            int p0, int nl) {
#pragma unroll
    for (int c = 0; c < Gm::CH; ++c) {
        const int ch = place_channel<Gm>(p0 + c * Gm::CL);
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (ch < tl.kleft && nl * 4 < N) {
            const float* q = p + (size_t)(tl.c0 + ch) * N + nl * 4;
            if (vec) VecIO<float, 4>::load(f, q);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (nl * 4 + i < N) f[i] = q[i];
        }
        if (RATE)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = decay_rate(f[i]);
        s[c][0] = pack2(f[0], f[1]);
        s[c][1] = pack2(f[2], f[3]);
    }
}
// The state a sequence starts (or a gradient ends) with: p's, or 0 without p.
template <typename Gm>
__device__ __forceinline__ void load_given(f2 (&s)[Gm::CH][2], const float* p, const ScanArgs& a, const ScanTile& tl,
                                           int p0, int nl) {
    if (p) {
        load_states<Gm, false>(s, p + (size_t)tl.b * a.D_ * a.N, tl, a.N, a.state_vec, p0, nl);
    } else {
#pragma unroll
        for (int c = 0; c < Gm::CH; ++c) s[c][0] = s[c][1] = both2(0.f);
    }
}
template <typename Gm>
__device__ __forceinline__ void store_states(float* p, const f2 (&s)[Gm::CH][2], const ScanArgs& a, const ScanTile& tl,
                                             int p0, int nl) {
#pragma unroll
    for (int c = 0; c < Gm::CH; ++c) {
        const int ch = place_channel<Gm>(p0 + c * Gm::CL);
        if (ch >= tl.kleft || nl * 4 >= a.N) continue;
        float f[4];
        unpack2(s[c][0], f[0], f[1]);
        unpack2(s[c][1], f[2], f[3]);
        float* q = p + ((size_t)tl.b * a.D_ + tl.c0 + ch) * a.N + nl * 4;
        if (a.state_vec) VecIO<float, 4>::store(q, f);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (nl * 4 + i < a.N) q[i] = f[i];
    }
}

// A helper thread's own slots in shared memory for the rows on their way, two
// steps of them: asynchronous copies complete in order, so a step waits for its
// own rows only. (Two sets of registers did not serve: a wait for the older
// loads waited for the newer ones too.) A RawVec<T, V> per vector.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
// vec: kWhole vectors or kPairs of elements are aligned to their size, or only
// elements are. Copies are of 4 bytes at least, so single bf16 elements take
// plain loads (slot_load, then slot_store once all loads of a step are under way).
// The forward kernels have an instance for whole vectors throughout: the other
// forms' code cost it 3% (the backward one nothing).
enum { kSingle = 0, kWhole = 1, kPairs = 2 };
template <typename T> __device__ __forceinline__ bool copies_fit(int vec) { return sizeof(T) == 4 || vec != kSingle; }

template <typename T, int V>
__device__ __forceinline__ void slot_fetch(uint32_t* slot, const T* p, bool on, int left, int vec) {
    if (on && vec == kWhole) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(slot)), "l"(p), "n"(V * (int)sizeof(T))
                     : "memory");
        return;
    }
    constexpr int kPer = 4 / sizeof(T);  // elements of a word
#pragma unroll
    for (int i = 0; i < RawVec<T, V>::kWords; ++i) {
        if (on && i * kPer < left)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slot + i)), "l"(p + i * kPer)
                         : "memory");
        else slot[i] = 0;
    }
}
template <typename T, int V> __device__ __forceinline__ RawVec<T, V> slot_load(const T* p, bool on, int left) {
    RawVec<T, V> r;
    r.zero();
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (on && j < left) r.set(j, p[j]);
    return r;
}
template <typename T, int V> __device__ __forceinline__ void slot_store(uint32_t* slot, const RawVec<T, V>& r) {
#pragma unroll
    for (int i = 0; i < RawVec<T, V>::kWords; ++i) slot[i] = r.w[i];
}
template <typename T, int V> __device__ __forceinline__ RawVec<T, V> slot_read(const uint32_t* slot) {
    RawVec<T, V> r;
    if constexpr (RawVec<T, V>::kWords == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (RawVec<T, V>::kWords == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(slot);
        r.w[0] = v.x; r.w[1] = v.y;
    } else {
        r.w[0] = slot[0];
    }
    return r;
}

// [L tokens][CB channels] of one input among the helpers: vector i of thread
// `ht` is number v = 128 i + ht, token v / VPT, channels from (v % VPT) VW (the
// same for every i). Tokens from n on and channels beyond the tile are not read
// and give 0.
template <typename T, typename Gm, int L> struct TokenRows {
    static constexpr int VW = Gm::VW, VPT = Gm::VPT, kAll = L * VPT;
    static constexpr int NV = kAll > kHelperThreads ? kAll / kHelperThreads : 1;
    static constexpr int kVec = RawVec<T, VW>::kWords;
    static constexpr int kWords = (kAll < kHelperThreads ? kAll : NV * kHelperThreads) * kVec;  // of a step's slots
    RawVec<T, VW> v[NV];
    static __device__ __forceinline__ int token(int i, int ht) { return (kHelperThreads * i + ht) / VPT; }
    static __device__ __forceinline__ int channel(int ht) { return ht % VPT * VW; }
    static __device__ __forceinline__ void fetch(uint32_t* slots, const T* p, long long st, int t0, const ScanTile& tl,
                                                 int vec, int ht) {
        const int ch = channel(ht);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int tok = token(i, ht);
            if (tok >= L) continue;
            slot_fetch<T, VW>(slots + (kHelperThreads * i + ht) * kVec, p + (t0 + tok) * st + ch,
                              t0 + tok < tl.n && ch < tl.kleft, tl.kleft - ch, vec);
        }
    }
    // the same with plain loads: first all inputs' loads, then the stores
    __device__ __forceinline__ void load(const T* p, long long st, int t0, const ScanTile& tl, int ht) {
        const int ch = channel(ht);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int tok = token(i, ht);
            v[i] = slot_load<T, VW>(p + (t0 + tok) * st + ch, tok < L && t0 + tok < tl.n && ch < tl.kleft, tl.kleft - ch);
        }
    }
    __device__ __forceinline__ void store(uint32_t* slots, int ht) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (token(i, ht) < L) slot_store<T, VW>(slots + (kHelperThreads * i + ht) * kVec, v[i]);
    }
    __device__ __forceinline__ void read(const uint32_t* slots, int ht) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i].zero();
            if (token(i, ht) < L) v[i] = slot_read<T, VW>(slots + (kHelperThreads * i + ht) * kVec);
        }
    }
};
template <typename T, int VW> __device__ __forceinline__ void store_row(T* p, const float (&f)[VW], int left, int vec) {
    if (vec) VecIO<T, VW>::store(p, f);
    else
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (j < left) p[j] = from_f32<T>(f[j]);
}

// [L tokens][N states] of B and of C behind it, staged as fp32 rows of NP.
template <typename T, typename Gm, int L> struct StateRows {
    static constexpr int kEach = L * Gm::NS, kAll = 2 * kEach;
    static constexpr int NV = kAll > kHelperThreads ? kAll / kHelperThreads : 1;
    static constexpr int kVec = RawVec<T, 4>::kWords;
    static constexpr int kWords = (kAll < kHelperThreads ? kAll : NV * kHelperThreads) * kVec;
    // vector i of a thread: where it is read from (null: nowhere) and how many states are left
    struct Source { const T* p; bool any, on; int left; };
    static __device__ __forceinline__ Source source(int i, const T* Bp, const T* Cp, const ScanArgs& a, int t0,
                                                    const ScanTile& tl, int ht) {
        const int e = kHelperThreads * i + ht, r = e % kEach, tok = r / Gm::NS, n0 = r % Gm::NS * 4;
        const T* p = e < kEach ? Bp : Cp;
        return {p + (t0 + tok) * (e < kEach ? a.bs[1] : a.cs[1]) + n0, e < kAll && p, t0 + tok < tl.n && n0 < a.N, a.N - n0};
    }
    static __device__ __forceinline__ void fetch(uint32_t* slots, const T* Bp, const T* Cp, const ScanArgs& a, int t0,
                                                 const ScanTile& tl, int vec, int ht) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Source s = source(i, Bp, Cp, a, t0, tl, ht);
            uint32_t* slot = slots + (kHelperThreads * i + ht) * kVec;
            if (s.any && copies_fit<T>(vec)) slot_fetch<T, 4>(slot, s.p, s.on, s.left, vec);
        }
        if (copies_fit<T>(vec)) return;
        constexpr int kTogether = NV < 4 ? NV : 4;
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += kTogether) {
            RawVec<T, 4> v[kTogether];
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                const Source s = source(i0 + i, Bp, Cp, a, t0, tl, ht);
                v[i] = slot_load<T, 4>(s.p, s.any && s.on, s.left);
            }
#pragma unroll
            for (int i = 0; i < kTogether; ++i)
                if (source(i0 + i, Bp, Cp, a, t0, tl, ht).any)
                    slot_store<T, 4>(slots + (kHelperThreads * (i0 + i) + ht) * kVec, v[i]);
        }
    }
    static __device__ __forceinline__ void stage(const uint32_t* slots, float* s, int ht, bool with_c) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = kHelperThreads * i + ht;
            if (e >= (with_c ? kAll : kEach)) continue;
            const RawVec<T, 4> v = slot_read<T, 4>(slots + e * kVec);
            const f2 q[2] = {pack2(v.get(0), v.get(1)), pack2(v.get(2), v.get(3))};
            sts_quad(s + 4 * e, q);
        }
    }
};

template <typename T, int VW> __device__ __forceinline__ void raw_floats(float (&f)[VW], const RawVec<T, VW>& r) {
#pragma unroll
    for (int i = 0; i < VW; ++i) f[i] = r.get(i);
}
// dt of raw steps, and (SIG) its derivative.
template <bool SIG, int VW>
__device__ __forceinline__ void step_sizes(float (&dt)[VW], float (&sig)[VW], const float (&raw)[VW], int softplus) {
#pragma unroll
    for (int i = 0; i < VW; i += 2) {
        StepCurve c = {pack2(raw[i], raw[i + 1]), both2(1.f)};
        if (softplus) c = softplus2<SIG>(c.dt);
        unpack2(c.dt, dt[i], dt[i + 1]);
        if (SIG) unpack2(c.sig, sig[i], sig[i + 1]);
    }
}
// Channels' values from a [D] array, 0 where absent.
template <int VW>
__device__ __forceinline__ void channel_values(float (&f)[VW], const float* p, const ScanTile& tl, int ch) {
#pragma unroll
    for (int j = 0; j < VW; ++j) f[j] = p && ch + j < tl.kleft ? p[tl.c0 + ch + j] : 0.f;
}

// Partial sums over the states: lanes whose numbers differ in bits above the
// lowest two are added here, the rest (NQ per channel, adjacent) by the reader.
template <typename Gm> __device__ __forceinline__ float fold_states(float v) {
#pragma unroll
    for (int m = 4; m < Gm::NS; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}
template <typename Gm> __device__ __forceinline__ float sum_states(const float* p) {
    if constexpr (Gm::NQ == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        return (v.x + v.y) + (v.z + v.w);
    } else if constexpr (Gm::NQ == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        return v.x + v.y;
    } else {
        return p[0];
    }
}

// Folds the maps state -> P state + h of the chunks [from, to) (step 1 or -1) of
// a walker's channels into s. Maps: [unit][chunk][walker][P, h].
template <typename Gm>
__device__ __forceinline__ void fold_chunks(f2 (&s)[Gm::CH][2], const float* ends, const ScanArgs& a,
                                            const ScanTile& tl, int walker, int lane, int from, int to, int step) {
    for (int c = from; step > 0 ? c < to : c > to; c += step) {
        const float* p = ends + ((tl.unit * a.chunks + c) * kWalkers + walker) * 2 * Gm::QUADS + lane * 4;
#pragma unroll
        for (int i = 0; i < Gm::CH; ++i) {
            f2 pw[2], hw[2];
            lds_quad(pw, p + i * 128);
            lds_quad(hw, p + Gm::QUADS + i * 128);
            s[i][0] = fma2(pw[0], s[i][0], hw[0]);
            s[i][1] = fma2(pw[1], s[i][1], hw[1]);
        }
    }
}
template <typename Gm>
__device__ __forceinline__ void store_map(float* ends, const f2 (&p)[Gm::CH][2], const f2 (&h)[Gm::CH][2],
                                          const ScanArgs& a, const ScanTile& tl, int walker, int lane) {
    float* o = ends + ((tl.unit * a.chunks + tl.part) * kWalkers + walker) * 2 * Gm::QUADS + lane * 4;
#pragma unroll
    for (int i = 0; i < Gm::CH; ++i) {
        sts_quad(o + i * 128, p[i]);
        sts_quad(o + Gm::QUADS + i * 128, h[i]);
    }
}

// Lanes that share a channel's states, by the state size.
inline int scan_lanes(int N) {
    int ns = 1;
    while (4 * ns < N) ns *= 2;
    return ns;
}
// Blocks' tiles of a group's K channels, at CH channels a lane.
inline int scan_tiles(int K, int N, int CH) {
    const int cb = kWalkers * CH * 32 / scan_lanes(N);
    return (K + cb - 1) / cb;
}

}  // namespace gdr
