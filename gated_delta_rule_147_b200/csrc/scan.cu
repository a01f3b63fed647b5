// Selective state-space scan: forward over whole sequences (also the backward
// pass's state checkpoints) and one token per sequence.
//
// The forward's floor is its exponentials: N per token and channel, and two with
// a reciprocal for softplus and gate, at 16 per clock and SM, against 6 to 8
// bytes of HBM traffic. Per pair of states and token a walker does dt A, exp2
// (twice), dt u B, h and C h in packed fp32.
//
// Where the channels alone leave SMs empty the tokens are split into chunks:
// one launch finds each chunk's map of its start state (decay and end from
// zero), and the second, whose blocks fold the maps before theirs, does the
// rest. That computes the exponentials twice, so it takes three chunks at least.
#include <type_traits>

#include "scan_common.cuh"

namespace gdr {

enum { kScanOut = 0, kScanEnds = 1, kScanCkpt = 2 };  // y; chunk maps; states every Seg tokens

// Words of shared memory: two steps of inputs (dt, dt u; B, C) and of sums, and
// of rows on their way (delta, u, z; B and C).
template <typename T, typename Gm, bool OUT> struct ScanFwdShared {
    static constexpr int LT = Gm::LT;
    static constexpr int in = 4 * LT * Gm::CB + 2 * LT * Gm::NP, out = OUT ? LT * Gm::CB * Gm::NQ : 0;
    using Rows = TokenRows<T, Gm, LT>;
    using States = StateRows<T, Gm, LT>;
    static constexpr int slots = 3 * Rows::kWords + States::kWords, total = 2 * (in + out + slots);
};

// Where a split forward chunk's fold starts: the first launch goes through chunk
// 0 from h0 itself and leaves h0 in the place of that chunk's decay, so that the
// second launch, which writes h_T (it may be h0), does not read h0.
template <typename Gm>
__device__ __forceinline__ void load_first(f2 (&s)[Gm::CH][2], const ScanArgs& a, const ScanTile& tl, int walker,
                                           int lane) {
    const float* p = a.ends + (tl.unit * a.chunks * kWalkers + walker) * 2 * Gm::QUADS + lane * 4;
#pragma unroll
    for (int c = 0; c < Gm::CH; ++c) lds_quad(s[c], p + (tl.part ? Gm::QUADS : 0) + c * 128);
}

template <typename T, typename Gm, int MODE, bool WHOLE>
__global__ void __launch_bounds__(kScanThreads, Gm::CH == 2 ? kFwdBlocks : 2 * kFwdBlocks) scan_fwd_kernel(ScanArgs a) {
    constexpr int CH = Gm::CH, LT = Gm::LT, CB = Gm::CB, CL = Gm::CL, NP = Gm::NP;
    using Sh = ScanFwdShared<T, Gm, MODE == kScanOut>;
    constexpr int kIn = Sh::in, kOut = Sh::out;
    extern __shared__ __align__(16) float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ScanTile tl(a, CB);
    if (MODE == kScanEnds && tl.part + 1 == a.chunks) return;  // no chunk after it
    const int steps = (tl.n - tl.t0 + LT - 1) / LT;
    float* const out = sm + 2 * kIn;

    if (warp < kWalkers) {
        const int nl = lane % Gm::NS, cl = lane / Gm::NS, p0 = lane_place<Gm>(warp, 0, cl);
        f2 A[CH][2], h[CH][2];
        load_states<Gm, true>(A, a.A, tl, a.N, a.state_vec, p0, nl);
        if (MODE == kScanOut && a.chunks > 1) {
            load_first<Gm>(h, a, tl, warp, lane);
            fold_chunks<Gm>(h, a.ends, a, tl, warp, lane, 1, tl.part, 1);
        } else {
            load_given<Gm>(h, MODE == kScanEnds && tl.part ? nullptr : a.h0, a, tl, p0, nl);
            if (MODE == kScanCkpt) fold_chunks<Gm>(h, a.ends, a, tl, warp, lane, 0, tl.part, 1);
        }
        f2 first[CH][2];
        if (MODE == kScanEnds)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                first[c][0] = h[c][0];
                first[c][1] = h[c][1];
            }
        f2 total[CH];  // sum of dt
        if (MODE == kScanEnds)
#pragma unroll
            for (int c = 0; c < CH; ++c) total[c] = both2(0.f);
        __syncthreads();
        for (int s = 0; s <= steps; ++s) {
            if (s < steps) {
                const float* in = sm + (s & 1) * kIn + p0 * 4;
                const float* B0 = sm + (s & 1) * kIn + 4 * LT * CB + 4 * nl;
                float* o = out + (s & 1) * kOut + p0 * Gm::NQ + nl;
                // a token's operands are loaded before the last one's sums are stored:
                // the compiler cannot tell that the two do not overlap
                struct { f2 B[2], C[2], d[CH][2]; } x, next;  // d: dt, dt u
                auto load = [&](decltype(x)& v, int t) {
                    lds_quad(v.B, B0 + t * NP);
                    if (MODE == kScanOut) lds_quad(v.C, B0 + (LT + t) * NP);
#pragma unroll
                    for (int c = 0; c < CH; ++c) lds_quad(v.d[c], in + (t * CB + c * CL) * 4);
                };
                load(x, 0);
#pragma unroll 1
                for (int tb = 0; tb < LT; tb += Gm::Seg) {
                    if (MODE == kScanCkpt) {
                        float* ck = a.ckpt + ((tl.unit * kWalkers + warp) * a.segs + (tl.t0 + s * LT + tb) / Gm::Seg) *
                                                 Gm::QUADS + lane * 4;
                        if (tl.t0 + s * LT + tb < tl.n)
#pragma unroll
                            for (int c = 0; c < CH; ++c) sts_quad(ck + c * 128, h[c]);
                    }
#pragma unroll
                    for (int i = 0; i < Gm::Seg; ++i) {
                        const int t = tb + i;
                        load(next, min(t + 1, LT - 1));
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                h[c][k] = fma2(decay2(x.d[c][0], A[c][k]), h[c][k], mul2(x.d[c][1], x.B[k]));
                            if (MODE == kScanEnds) total[c] = add2(total[c], x.d[c][0]);
                            if (MODE == kScanOut) {
                                const float v = fold_states<Gm>(sum2(fma2(x.C[1], h[c][1], mul2(x.C[0], h[c][0]))));
                                if (nl < Gm::NQ) o[(t * CB + c * CL) * Gm::NQ] = v;
                            }
                        }
                        x = next;
                    }
                }
            }
            __syncthreads();
        }
        if (MODE == kScanEnds) {
            f2 p[CH][2];
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k) p[c][k] = tl.part ? ex2_pair(mul2(total[c], A[c][k])) : first[c][k];
            store_map<Gm>(a.ends, p, h, a, tl, warp, lane);
        }
        const int last = max(seq_len(a.lengths, tl.b, a.T) - 1, 0) / a.chunk;
        if (MODE == kScanOut && a.h_T && tl.part == last) store_states<Gm>(a.h_T, h, a, tl, p0, nl);
    } else {
        const int ht = threadIdx.x - 32 * kWalkers;
        const T* u = reinterpret_cast<const T*>(a.u) + tl.b * a.us[0] + tl.c0;
        const T* dl = reinterpret_cast<const T*>(a.delta) + tl.b * a.ds[0] + tl.c0;
        const T* z = MODE == kScanOut && a.z ? reinterpret_cast<const T*>(a.z) + tl.b * a.zs[0] + tl.c0 : nullptr;
        const T* Bm = reinterpret_cast<const T*>(a.Bm) + tl.b * a.bs[0] + tl.g * a.N;
        const T* Cm = MODE == kScanOut ? reinterpret_cast<const T*>(a.Cm) + tl.b * a.cs[0] + tl.g * a.N : nullptr;
        using Rows = typename Sh::Rows;
        constexpr int VW = Rows::VW;
        const int vch = Rows::channel(ht);
        T* y = reinterpret_cast<T*>(a.y) + (size_t)tl.b * a.T * a.D_ + tl.c0 + vch;
        using States = typename Sh::States;
        const int rows = WHOLE ? (int)kWhole : a.act_vec, vecs = WHOLE ? (int)kWhole : a.bc_vec;
        Rows held_u[2], held_z[2];  // of the steps staged and walked
        uint32_t* const slots = reinterpret_cast<uint32_t*>(out + 2 * kOut);
        float bias[VW], skip[VW];
        channel_values(bias, a.bias, tl, vch);
        channel_values(skip, a.D, tl, vch);
        auto fetch = [&](int s) {  // into the slots of step s - 2
            uint32_t* w = slots + (s & 1) * Sh::slots;
            if (s < steps) {
                const int t0 = tl.t0 + s * LT;
                if (copies_fit<T>(rows)) {
                    Rows::fetch(w, dl, a.ds[1], t0, tl, rows, ht);
                    Rows::fetch(w + Rows::kWords, u, a.us[1], t0, tl, rows, ht);
                    if (z) Rows::fetch(w + 2 * Rows::kWords, z, a.zs[1], t0, tl, rows, ht);
                } else {
                    Rows r[3];
                    r[0].load(dl, a.ds[1], t0, tl, ht);
                    r[1].load(u, a.us[1], t0, tl, ht);
                    if (z) r[2].load(z, a.zs[1], t0, tl, ht);
                    r[0].store(w, ht);
                    r[1].store(w + Rows::kWords, ht);
                    if (z) r[2].store(w + 2 * Rows::kWords, ht);
                }
                States::fetch(w + 3 * Rows::kWords, Bm, Cm, a, t0, tl, vecs, ht);
            }
            copies_commit();
        };
        auto stage = [&](int s) {
            held_u[0] = held_u[1];
            held_z[0] = held_z[1];
            copies_wait<1>();
            if (s < steps) {
                float* in = sm + (s & 1) * kIn;
                const uint32_t* w = slots + (s & 1) * Sh::slots;
                Rows rd;
                rd.read(w, ht);
                held_u[1].read(w + Rows::kWords, ht);
                if (z) held_z[1].read(w + 2 * Rows::kWords, ht);
#pragma unroll
                for (int i = 0; i < Rows::NV; ++i) {
                    const int tok = Rows::token(i, ht);
                    const bool on = tl.t0 + s * LT + tok < tl.n && vch < tl.kleft;
                    float raw[VW], uf[VW], dt[VW];
                    raw_floats(raw, rd.v[i]);
                    raw_floats(uf, held_u[1].v[i]);
#pragma unroll
                    for (int j = 0; j < VW; ++j) raw[j] += bias[j];
                    step_sizes<false>(dt, dt, raw, a.softplus);
                    if (tok < LT)
#pragma unroll
                        for (int j = 0; j < VW; ++j) {
                            const float d = on ? dt[j] : 0.f;
                            const f2 q[2] = {both2(d), both2(d * uf[j])};
                            sts_quad(in + (tok * CB + channel_place<Gm>(vch + j)) * 4, q);
                        }
                }
                States::stage(w + 3 * Rows::kWords, in + 4 * LT * CB, ht, MODE == kScanOut);
            }
            fetch(s + 2);
        };
        fetch(0);
        fetch(1);
        stage(0);
        __syncthreads();
        for (int s = 0; s <= steps; ++s) {
            const Rows last_u = held_u[0], last_z = held_z[0];
            stage(s + 1);
            if (MODE == kScanOut && s > 0) {
                const float* o = out + ((s - 1) & 1) * kOut;
#pragma unroll
                for (int i = 0; i < Rows::NV; ++i) {
                    const int tok = Rows::token(i, ht), t = tl.t0 + (s - 1) * LT + tok;
                    if (tok >= LT || t >= tl.t1 || vch >= tl.kleft) continue;
                    float f[VW], uf[VW], zf[VW];
                    raw_floats(uf, last_u.v[i]);
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        f[j] = fmaf(skip[j], uf[j],
                                    sum_states<Gm>(o + (tok * CB + channel_place<Gm>(vch + j)) * Gm::NQ));
                    if (z) {
                        raw_floats(zf, last_z.v[i]);
#pragma unroll
                        for (int j = 0; j < VW; j += 2) {
                            const f2 zz = pack2(zf[j], zf[j + 1]);
                            unpack2(mul2(mul2(zz, sigmoid2(zz)), pack2(f[j], f[j + 1])), f[j], f[j + 1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        if (t >= tl.n) f[j] = 0.f;
                    store_row(y + (size_t)t * a.D_, f, tl.kleft - vch, a.out_vec);
                }
            }
            __syncthreads();
        }
    }
    if (MODE == kScanOut) {
        // rows from the last step on hold no token
        static_assert(kScanThreads % CB == 0, "whole rows of threads");
        const int ch = threadIdx.x % CB, t0 = min(tl.t1, tl.t0 + steps * LT);
        T* y = reinterpret_cast<T*>(a.y) + (size_t)tl.b * a.T * a.D_ + tl.c0 + ch;
        if (ch < tl.kleft)
            for (int t = t0 + threadIdx.x / CB; t < tl.t1; t += kScanThreads / CB) y[(size_t)t * a.D_] = from_f32<T>(0.f);
    }
}

template <typename T, int NS, int MODE> static cudaError_t launch_fwd_geom(const ScanArgs& a, int B, cudaStream_t st) {
    using Gm = std::conditional_t<MODE == kScanCkpt, ScanCkptGeom<NS>,
                                  std::conditional_t<MODE == kScanEnds, ScanEndsGeom<NS>, ScanFwdGeom<NS>>>;
    const long long grid = (long long)B * a.G * a.tiles * a.chunks;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    constexpr size_t smem = ScanFwdShared<T, Gm, MODE == kScanOut>::total * sizeof(float);
    static_assert(smem <= 227 * 1024, "shared memory of a block");
    const bool whole = a.act_vec == kWhole && a.bc_vec == kWhole;
    auto kern = whole ? scan_fwd_kernel<T, Gm, MODE, true> : scan_fwd_kernel<T, Gm, MODE, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)grid, kScanThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename F> static cudaError_t dispatch_scan_lanes(int ns, F&& f) {
    switch (ns) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 4: return f(std::integral_constant<int, 4>());
        case 8: return f(std::integral_constant<int, 8>());
        case 16: return f(std::integral_constant<int, 16>());
        default: return f(std::integral_constant<int, 32>());
    }
}

// Chunks of the tokens: as many as fill two blocks per SM, of 256 tokens at
// least, and none below three (see above). One sequence of 2048 channels x 16
// states in bf16: 768 tokens 37.5 us split and 58.7 whole, 4096 106 and 298. The
// 256 is not borne out for short sequences: with 64, 512 tokens would take 20.6 us
// where they now take 40.5, and 768 27.3; from 2048 on nothing changes.
int scan_chunks(int B, int T, int K, int N, int G) {
    const long long units = (long long)B * G * scan_tiles(K, N, 2);
    const long long c = units > 0 ? 148 * kFwdBlocks / units : 0, most = T / 256;
    const long long n = c < most ? c : most;
    return n < 3 ? 1 : (int)n;
}
// Sets the split; a chunk is a whole number of steps and segments.
void scan_split(ScanArgs& a, int chunks, int CH) {
    const int per = (a.T + chunks - 1) / chunks;
    a.chunk = per < 32 ? 32 : (per + 31) / 32 * 32;
    a.chunks = a.T > 0 ? (a.T - 1) / a.chunk + 1 : 1;
    a.tiles = scan_tiles(a.K, a.N, CH);
}
size_t scan_ends_bytes(int B, int G, int K, int N, int chunks, int CH) {
    return chunks < 2 ? 0 : (size_t)B * G * scan_tiles(K, N, CH) * chunks * kWalkers * 2 * CH * 128 * sizeof(float);
}

template <int MODE> static cudaError_t launch_fwd_mode(const ScanArgs& a, int B, int dtype, cudaStream_t st) {
    return dispatch_scan_lanes(scan_lanes(a.N), [&](auto nc) {
        constexpr int NS = decltype(nc)::value;
        return dtype == GDR_BF16 ? launch_fwd_geom<__nv_bfloat16, NS, MODE>(a, B, st)
                                 : launch_fwd_geom<float, NS, MODE>(a, B, st);
    });
}
cudaError_t launch_scan_fwd(const ScanArgs& a, int B, int dtype, cudaStream_t st) {
    if (a.chunks > 1) {
        cudaError_t e = launch_fwd_mode<kScanEnds>(a, B, dtype, st);
        if (e != cudaSuccess) return e;
    }
    return launch_fwd_mode<kScanOut>(a, B, dtype, st);
}
// The backward pass's checkpoints: the state at every segment's start.
cudaError_t launch_scan_ckpt(const ScanArgs& a, int B, int dtype, cudaStream_t st) {
    return launch_fwd_mode<kScanCkpt>(a, B, dtype, st);
}

// One token. Bound by HBM: 8 bytes per state, read and written once. A warp
// holds 32 channels of one (sequence, group): lane l does the per-channel work
// (softplus, gate, y) of channel l once, and the states go by in NS steps of
// 32 / NS channels, 4 adjacent states a lane, whose loads are all requested
// before the first is used (up to kStepAhead steps at a time).
// Steps ahead and blocks per SM, 256 sequences of 4096 channels x 16 states in
// bf16: 4 and 3 take 37.1 us, 4 and 4 33.0, 1 and 6 33.8, 2 and 5 29.6 (4.83 TB/s).
constexpr int kStepAhead = 2, kStepBlocks = 5;

template <typename T, int NS>
__global__ void __launch_bounds__(256, kStepBlocks) scan_step_kernel(ScanArgs a, float* h, unsigned warps) {
    dependent_launch();
    constexpr int CL = 32 / NS, kBatch = NS < kStepAhead ? NS : kStepAhead;
    const unsigned tile = blockIdx.x * 8 + threadIdx.x / 32;
    if (tile >= warps) return;
    const int lane = threadIdx.x & 31, nl = lane % NS, cl = lane / NS, n0 = 4 * nl;
    const unsigned r = tile / (unsigned)a.tiles;
    const int g = (int)(r % (unsigned)a.G), t = (int)(tile - r * a.tiles);
    const long long b = r / (unsigned)a.G;
    const int c0 = g * a.K + 32 * t, kleft = min(32, a.K - 32 * t);
    dependent_wait();
    const bool mine = n0 < a.N, own = lane < kleft;
    RawVec<T, 4> Br, Cr;
    Br.zero();
    Cr.zero();
    if (mine) {
        const T* Bp = reinterpret_cast<const T*>(a.Bm) + b * a.bs[0] + g * a.N + n0;
        const T* Cp = reinterpret_cast<const T*>(a.Cm) + b * a.cs[0] + g * a.N + n0;
        if (a.bc_vec == kWhole) {
            Br.load(Bp);
            Cr.load(Cp);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < a.N) { Br.set(i, Bp[i]); Cr.set(i, Cp[i]); }
        }
    }
    float uf = 0.f, raw = 0.f, zf = 0.f, skip = 0.f;
    if (own) {
        const int c = c0 + lane;
        uf = to_f32(reinterpret_cast<const T*>(a.u)[b * a.us[0] + c]);
        raw = to_f32(reinterpret_cast<const T*>(a.delta)[b * a.ds[0] + c]) + (a.bias ? a.bias[c] : 0.f);
        if (a.D) skip = a.D[c];
        if (a.z) zf = to_f32(reinterpret_cast<const T*>(a.z)[b * a.zs[0] + c]);
    }
    const float* Ap = a.A + (size_t)c0 * a.N + n0;
    float* hp = h + ((size_t)b * a.D_ + c0) * a.N + n0;
    float dt = 0.f, y = 0.f;
    const f2 B[2] = {pack2(Br.get(0), Br.get(1)), pack2(Br.get(2), Br.get(3))};
    const f2 C[2] = {pack2(Cr.get(0), Cr.get(1)), pack2(Cr.get(2), Cr.get(3))};
#pragma unroll 1
    for (int s0 = 0; s0 < NS; s0 += kBatch) {
        float s[kBatch][4], A[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int ch = (s0 + k) * CL + cl;
            const bool on = mine && ch < kleft;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[k][i] = A[k][i] = 0.f;
            if (on && a.state_vec) {
                VecIO<float, 4>::load(s[k], hp + ch * a.N);
                VecIO<float, 4>::load(A[k], Ap + ch * a.N);
            } else if (on) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < a.N) { s[k][i] = hp[ch * a.N + i]; A[k][i] = Ap[ch * a.N + i]; }
            }
        }
        if (s0 == 0) dt = !own ? 0.f : a.softplus ? softplusf(raw) : raw;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int ch = (s0 + k) * CL + cl;
            const float dtc = __shfl_sync(0xffffffffu, dt, ch), dtu = __shfl_sync(0xffffffffu, dt * uf, ch);
            f2 yv = both2(0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) A[k][i] = decay_rate(A[k][i]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f2 v = fma2(decay2(both2(dtc), pack2(A[k][2 * q], A[k][2 * q + 1])),
                            pack2(s[k][2 * q], s[k][2 * q + 1]), mul2(both2(dtu), B[q]));
                yv = fma2(C[q], v, yv);
                unpack2(v, s[k][2 * q], s[k][2 * q + 1]);
            }
            if (mine && ch < kleft) {
                if (a.state_vec) VecIO<float, 4>::store(hp + ch * a.N, s[k]);
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n0 + i < a.N) hp[ch * a.N + i] = s[k][i];
            }
            float v = sum2(yv);
#pragma unroll
            for (int m = NS / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            v = __shfl_sync(0xffffffffu, v, (lane % CL) * NS);  // to the channel's own lane
            if (lane / CL == s0 + k) y = v;
        }
    }
    if (own) {
        y = fmaf(skip, uf, y);
        if (a.z) y *= zf * sigmoidf_fast(zf);
        reinterpret_cast<T*>(a.y)[(size_t)b * a.D_ + c0 + lane] = from_f32<T>(y);
    }
}

cudaError_t launch_scan_step(ScanArgs a, float* h, int B, int dtype, cudaStream_t st) {
    return dispatch_scan_lanes(scan_lanes(a.N), [&](auto nc) {
        constexpr int NS = decltype(nc)::value;
        a.tiles = (a.K + 31) / 32;
        const long long warps = (long long)B * a.G * a.tiles, grid = (warps + 7) / 8;
        if (warps > 0x7fffffffll) return cudaErrorInvalidValue;
        return dtype == GDR_BF16
                   ? launch_dependent(scan_step_kernel<__nv_bfloat16, NS>, (unsigned)grid, 256, 0, st, a, h, (unsigned)warps)
                   : launch_dependent(scan_step_kernel<float, NS>, (unsigned)grid, 256, 0, st, a, h, (unsigned)warps);
    });
}

}  // namespace gdr
