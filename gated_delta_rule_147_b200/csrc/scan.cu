// Selective state-space scan: forward over whole sequences (also the backward
// pass's state checkpoints) and one token per sequence.
//
// The forward's floor is its exponentials: N per token and channel at 16 per
// clock and SM, against 6 to 8 bytes of HBM traffic. One pass computes each
// exponential once. Per pair of states and token, in packed fp32:
// dt A, exp2 (twice), dt u B, h, C h, and, so that a segment can start before
// its incoming state is known, the running decay p and C p. When the state
// arrives, y += (C p) h_in is one multiply-add, and the outgoing state
// p h_in + h goes on to the next warp before that.
#include <type_traits>

#include "scan_common.cuh"

namespace gdr {

template <typename T, typename Gm, bool CKPT>
__global__ void __launch_bounds__(kScanThreads) scan_fwd_kernel(ScanArgs a) {
    constexpr int CH = Gm::CH, L = Gm::L, CPW = Gm::CPW, NP = Gm::NP;
    extern __shared__ __align__(16) float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nl = lane % Gm::NS, cl = lane / Gm::NS;
    constexpr int kWarpFloats = 3 * L * CPW + 2 * L * NP;
    float* sdt = sm + warp * kWarpFloats;
    float* sdtu = sdt + L * CPW;
    float* sy = sdtu + L * CPW;
    float* sB = sy + L * CPW;
    float* sC = sB + L * NP;
    float* carry = sm + kScanWarps * kWarpFloats;  // [warp][CH][32] quads: the state a warp starts from
    const ScanTile tl(a, CPW);
    const T* u = reinterpret_cast<const T*>(a.u) + tl.b * a.us[0] + tl.c0;
    const T* dl = reinterpret_cast<const T*>(a.delta) + tl.b * a.ds[0] + tl.c0;
    const T* z = a.z ? reinterpret_cast<const T*>(a.z) + tl.b * a.zs[0] + tl.c0 : nullptr;
    const T* Bm = reinterpret_cast<const T*>(a.Bm) + tl.b * a.bs[0] + tl.g * a.N;
    const T* Cm = reinterpret_cast<const T*>(a.Cm) + tl.b * a.cs[0] + tl.g * a.N;
    T* y = reinterpret_cast<T*>(a.y) + (size_t)tl.b * a.T * a.D_ + tl.c0;
    const size_t sbase = (size_t)tl.b * a.D_ * a.N;
    const int nseg = (tl.n + L - 1) / L;

    f2 A[CH][2];
    load_states<Gm>(A, a.A, tl, a.N, a.state_vec, cl, nl, kLog2e, true);
    // a lane's staged elements keep their channel from segment to segment
    float bias[Gm::SE], skip[Gm::SE];
#pragma unroll
    for (int i = 0; i < Gm::SE; ++i) {
        const int ch = (32 * i + lane) % CPW;
        bias[i] = a.bias && ch < tl.kleft ? a.bias[tl.c0 + ch] : 0.f;
        skip[i] = !CKPT && a.D && ch < tl.kleft ? a.D[tl.c0 + ch] : 0.f;
    }
    T ru[Gm::SE], rd[Gm::SE], rz[Gm::SE], rB[Gm::BE], rC[Gm::BE];
    auto fetch = [&](int seg) {
        fetch_rows<T, Gm>(ru, u, a.us[1], seg * L, tl, lane);
        fetch_rows<T, Gm>(rd, dl, a.ds[1], seg * L, tl, lane);
        fetch_vecs<T, Gm>(rB, Bm, a.bs[1], seg * L, tl, a.N, lane);
        if constexpr (!CKPT) {
            if (z) fetch_rows<T, Gm>(rz, z, a.zs[1], seg * L, tl, lane);
            fetch_vecs<T, Gm>(rC, Cm, a.cs[1], seg * L, tl, a.N, lane);
        }
    };
    if (warp < nseg) fetch(warp);
    for (int seg = warp; seg < nseg; seg += kScanWarps) {
        float du[Gm::SE], gate[Gm::SE];  // D u and silu(z) of the staged elements
#pragma unroll
        for (int i = 0; i < Gm::SE; ++i) {
            const int e = 32 * i + lane, step = e / CPW, ch = e % CPW;
            const bool on = seg * L + step < tl.n && ch < tl.kleft;
            const float uf = to_f32(ru[i]), raw = to_f32(rd[i]) + bias[i];
            const float dt = !on ? 0.f : a.softplus ? softplusf_series(raw) : raw;
            if (step < L) {
                sdt[e] = dt;
                sdtu[e] = dt * uf;
            }
            du[i] = skip[i] * uf;
            gate[i] = 1.f;
            if (!CKPT && z) {
                const float zf = to_f32(rz[i]);
                gate[i] = zf * sigmoidf_fast(zf);
            }
        }
        stage_vecs<T, Gm>(sB, rB, lane);
        if constexpr (!CKPT) stage_vecs<T, Gm>(sC, rC, lane);
        __syncwarp();
        if (seg + kScanWarps < nseg) fetch(seg + kScanWarps);

        f2 h[CH][2], p[CH][2];
        f2 yv[CKPT ? 1 : L][CH], q[CKPT ? 1 : L][CH][2];
#pragma unroll
        for (int t = 0; t < L; ++t) {
            f2 B[2], C[2];
            lds_quad(B, sB + t * NP + 4 * nl);
            if constexpr (!CKPT) lds_quad(C, sC + t * NP + 4 * nl);
            float dt[CH], dtu[CH];
            lds_run<CH>(dt, sdt + t * CPW + cl * CH);
            lds_run<CH>(dtu, sdtu + t * CPW + cl * CH);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const f2 dt2 = pack2(dt[c], dt[c]), dtu2 = pack2(dtu[c], dtu[c]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 dec = ex2_pair(mul2(dt2, A[c][k]));
                    const f2 in = mul2(dtu2, B[k]);
                    h[c][k] = t == 0 ? in : fma2(dec, h[c][k], in);
                    p[c][k] = t == 0 ? dec : mul2(p[c][k], dec);
                    if constexpr (!CKPT) {
                        yv[t][c] = k == 0 ? mul2(C[k], h[c][k]) : fma2(C[k], h[c][k], yv[t][c]);
                        q[t][c][k] = mul2(C[k], p[c][k]);
                    }
                }
            }
        }
        // the state before this segment
        f2 in[CH][2];
        if (seg == 0) {
            if (a.h0) load_states<Gm>(in, a.h0 + sbase, tl, a.N, a.state_vec, cl, nl, 1.f, false);
            else
#pragma unroll
                for (int c = 0; c < CH; ++c) in[c][0] = in[c][1] = pack2(0.f, 0.f);
        } else {
            carry_wait(warp);
#pragma unroll
            for (int c = 0; c < CH; ++c) lds_quad(in[c], carry + warp * Gm::QUADS + (c * 32 + lane) * 4);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k) h[c][k] = fma2(p[c][k], in[c][k], h[c][k]);
        if (seg + 1 < nseg) {
            const int to = (warp + 1) % kScanWarps;
#pragma unroll
            for (int c = 0; c < CH; ++c) sts_quad(carry + to * Gm::QUADS + (c * 32 + lane) * 4, h[c]);
            carry_arrive(to);
        } else if (!CKPT && a.h_T) {
            store_states<Gm>(a.h_T + sbase, h, tl, a.N, a.state_vec, cl, nl);
        }
        if constexpr (CKPT) {
            float* ck = a.ckpt + ((size_t)blockIdx.x * a.nseg + seg) * Gm::QUADS;
#pragma unroll
            for (int c = 0; c < CH; ++c) sts_quad(ck + (c * 32 + lane) * 4, in[c]);
        } else {
#pragma unroll
            for (int t = 0; t < L; ++t) {
                float v[CH];
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    f2 s = fma2(q[t][c][0], in[c][0], yv[t][c]);
                    s = fma2(q[t][c][1], in[c][1], s);
                    v[c] = sum2(s);
                }
                using Sum = LaneSum<CH, Gm::NS, 1>;
                Sum::run(v, nl);
                if (Sum::owner(nl)) {
#pragma unroll
                    for (int i = 0; i < Sum::left(); ++i) sy[t * CPW + cl * CH + Sum::first(nl) + i] = v[i];
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < Gm::SE; ++i) {
                const int e = 32 * i + lane, step = e / CPW, ch = e % CPW, t = seg * L + step;
                if (step < L && t < a.T && ch < tl.kleft)
                    y[(size_t)t * a.D_ + ch] = from_f32<T>(t < tl.n ? (sy[e] + du[i]) * gate[i] : 0.f);
            }
        }
        __syncwarp();
    }
    if constexpr (!CKPT) {
        // rows from the last segment on hold no token
        for (int e = threadIdx.x; e < (a.T - min(a.T, nseg * L)) * CPW; e += kScanThreads) {
            const int t = nseg * L + e / CPW, ch = e % CPW;
            if (ch < tl.kleft) y[(size_t)t * a.D_ + ch] = from_f32<T>(0.f);
        }
        if (nseg == 0 && warp == 0 && a.h_T) {
            f2 in[CH][2];
            if (a.h0) load_states<Gm>(in, a.h0 + sbase, tl, a.N, a.state_vec, cl, nl, 1.f, false);
            else
#pragma unroll
                for (int c = 0; c < CH; ++c) in[c][0] = in[c][1] = pack2(0.f, 0.f);
            store_states<Gm>(a.h_T + sbase, in, tl, a.N, a.state_vec, cl, nl);
        }
    }
}

template <typename T, typename Gm, bool CKPT> static cudaError_t launch_fwd_geom(ScanArgs a, int B, cudaStream_t st) {
    a.tiles = (a.K + Gm::CPW - 1) / Gm::CPW;
    const long long grid = (long long)B * a.G * a.tiles;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    const size_t smem = (size_t)kScanWarps * (3 * Gm::L * Gm::CPW + 2 * Gm::L * Gm::NP + Gm::QUADS) * sizeof(float);
    auto kern = scan_fwd_kernel<T, Gm, CKPT>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
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

cudaError_t launch_scan_fwd(const ScanArgs& a, int B, int dtype, cudaStream_t st) {
    return dispatch_scan_lanes(scan_lanes(a.N), [&](auto nc) {
        constexpr int NS = decltype(nc)::value;
        using Gm = ScanGeom<NS, NS == 1 ? 2 : 4, 4>;
        return dtype == GDR_BF16 ? launch_fwd_geom<__nv_bfloat16, Gm, false>(a, B, st)
                                 : launch_fwd_geom<float, Gm, false>(a, B, st);
    });
}

// The backward pass's first launch: the state at the start of every segment of
// its geometry (2 channels per lane, 8 tokens).
cudaError_t launch_scan_ckpt(const ScanArgs& a, int B, int dtype, cudaStream_t st) {
    return dispatch_scan_lanes(scan_lanes(a.N), [&](auto nc) {
        constexpr int NS = decltype(nc)::value;
        using Gm = ScanGeom<NS, 2, 8>;
        return dtype == GDR_BF16 ? launch_fwd_geom<__nv_bfloat16, Gm, true>(a, B, st)
                                 : launch_fwd_geom<float, Gm, true>(a, B, st);
    });
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
        if (a.bc_vec) {
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
        if (s0 == 0) dt = !own ? 0.f : a.softplus ? softplusf_series(raw) : raw;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int ch = (s0 + k) * CL + cl;
            const float dtc = __shfl_sync(0xffffffffu, dt, ch), dtu = __shfl_sync(0xffffffffu, dt * uf, ch);
            f2 yv = both2(0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) A[k][i] = fmaxf(A[k][i] * kLog2e, -3.402823466e38f);  // as load_states
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f2 v = fma2(ex2_pair(mul2(both2(dtc), pack2(A[k][2 * q], A[k][2 * q + 1]))),
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
