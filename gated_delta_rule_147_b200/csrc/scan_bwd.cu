// Selective state-space scan: backward pass.
//
// With g_t = dL/dh_t, yh = y before the gate and dyh = dy z sigmoid(z):
//   g_t = C_t dyh_t + a_{t+1} g_{t+1},  a = exp(dt A);   dh0 = a_1 g_1
//   dC_t = sum_d dyh h_t,  dB_t = sum_d dt u g_t
//   du = dt sum_n g B + D dyh,  d dt = sum_n g (u B + A a h_{t-1})
//   dA = sum dt a g h_{t-1},  dD = sum dyh u,  dz = dy yh (z sigmoid(z))'
//   ddelta = d dt sigmoid(delta + bias) (with softplus).
// Three launches. The forward scan first stores the state at every segment's
// start (scan.cu). The second walks the segments from the last to the first:
// a warp rebuilds its segment's states from the stored one (kept in
// registers) and, with the running decay p, its own contribution to the
// outgoing state gradient, sum_t p_t C_t dyh_t; the incoming one is then one
// multiply-add away from the next warp, and the segment is walked back with
// its decays recomputed (cheaper than holding them: the exponentials run beside
// the multiply-adds that bound this kernel). dB and dC are summed over a warp's
// channels by a shuffle reduction; the third launch adds the channel tiles, and
// the sequences' parameter gradients, in a fixed order.
#include <type_traits>

#include "scan_common.cuh"

namespace gdr {

constexpr float kLn2 = 0.6931471805599453f;

template <typename T, typename TG, typename Gm>
__global__ void __launch_bounds__(kScanThreads, 1) scan_bwd_kernel(ScanArgs a) {
    constexpr int CH = Gm::CH, L = Gm::L, CPW = Gm::CPW, NP = Gm::NP, NS = Gm::NS;
    static_assert(CH == 2, "channels of a lane");
    extern __shared__ __align__(16) float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nl = lane % NS, cl = lane / NS;
    constexpr int kRows = 6;  // dt, dt u, dyh; sums of C h, g B, A a g h
    constexpr int kWarpFloats = kRows * L * CPW + 2 * L * NP;
    float* sdt = sm + warp * kWarpFloats;
    float* sdtu = sdt + L * CPW;
    float* sdy = sdtu + L * CPW;
    float* sY = sdy + L * CPW;
    float* sGB = sY + L * CPW;
    float* sDD = sGB + L * CPW;
    float* sB = sDD + L * CPW;
    float* sC = sB + L * NP;
    float* carry = sm + kScanWarps * kWarpFloats;
    const ScanTile tl(a, CPW);
    const T* u = reinterpret_cast<const T*>(a.u) + tl.b * a.us[0] + tl.c0;
    const T* dl = reinterpret_cast<const T*>(a.delta) + tl.b * a.ds[0] + tl.c0;
    const T* z = a.z ? reinterpret_cast<const T*>(a.z) + tl.b * a.zs[0] + tl.c0 : nullptr;
    const TG* dy = reinterpret_cast<const TG*>(a.dy) + tl.b * a.gs[0] + tl.c0;
    const T* Bm = reinterpret_cast<const T*>(a.Bm) + tl.b * a.bs[0] + tl.g * a.N;
    const T* Cm = reinterpret_cast<const T*>(a.Cm) + tl.b * a.cs[0] + tl.g * a.N;
    const size_t rbase = (size_t)tl.b * a.T * a.D_ + tl.c0, sbase = (size_t)tl.b * a.D_ * a.N;
    float* bcp = a.bcpart + (((size_t)tl.tile * (gridDim.x / (a.tiles * a.G)) + tl.b) * a.T * a.G + tl.g) * (2 * NP);
    const int nseg = (tl.n + L - 1) / L;

    f2 A[CH][2], dA[CH][2];
    load_states<Gm>(A, a.A, tl, a.N, a.state_vec, cl, nl, kLog2e, true);
#pragma unroll
    for (int c = 0; c < CH; ++c) dA[c][0] = dA[c][1] = pack2(0.f, 0.f);
    constexpr int AC = CPW > 32 ? CPW / 32 : 1;  // channels of a lane's staged elements
    float bias[AC], skip[AC], dD[AC], db[AC];
#pragma unroll
    for (int i = 0; i < AC; ++i) {
        const int ch = (32 * i + lane) % CPW;
        bias[i] = a.bias && ch < tl.kleft ? a.bias[tl.c0 + ch] : 0.f;
        skip[i] = a.D && ch < tl.kleft ? a.D[tl.c0 + ch] : 0.f;
        dD[i] = db[i] = 0.f;
    }
    T ru[Gm::SE], rd[Gm::SE], rz[Gm::SE], rB[Gm::BE], rC[Gm::BE];
    TG rg[Gm::SE];
    auto fetch = [&](int seg) {
        fetch_rows<T, Gm>(ru, u, a.us[1], seg * L, tl, lane);
        fetch_rows<T, Gm>(rd, dl, a.ds[1], seg * L, tl, lane);
        if (z) fetch_rows<T, Gm>(rz, z, a.zs[1], seg * L, tl, lane);
        fetch_rows<TG, Gm>(rg, dy, a.gs[1], seg * L, tl, lane);
        fetch_vecs<T, Gm>(rB, Bm, a.bs[1], seg * L, tl, a.N, lane);
        fetch_vecs<T, Gm>(rC, Cm, a.cs[1], seg * L, tl, a.N, lane);
    };
    // warp w takes the segments nseg - 1 - w, nseg - 1 - w - kScanWarps, ...
    if (nseg - 1 - warp >= 0) fetch(nseg - 1 - warp);
    for (int seg = nseg - 1 - warp; seg >= 0; seg -= kScanWarps) {
        float uf[Gm::SE], sig[Gm::SE], gz[Gm::SE];  // u, ddt/ddelta, dy dgate/dz
        const float* ck = a.ckpt + ((size_t)blockIdx.x * a.nseg + seg) * Gm::QUADS;
        f2 h0[CH][2];
#pragma unroll
        for (int c = 0; c < CH; ++c) lds_quad(h0[c], ck + (c * 32 + lane) * 4);
#pragma unroll
        for (int i = 0; i < Gm::SE; ++i) {
            const int e = 32 * i + lane, step = e / CPW, ch = e % CPW;
            const bool on = seg * L + step < tl.n && ch < tl.kleft;
            uf[i] = to_f32(ru[i]);
            const float raw = to_f32(rd[i]) + bias[i % AC];
            const float dt = !on ? 0.f : a.softplus ? softplusf_series(raw) : raw;
            sig[i] = !on ? 0.f : a.softplus ? sigmoidf_fast(raw) : 1.f;
            float dyh = to_f32(rg[i]);
            gz[i] = 0.f;
            if (z) {
                const float zf = to_f32(rz[i]), sg = sigmoidf_fast(zf);
                gz[i] = on ? dyh * (sg * fmaf(zf, 1.f - sg, 1.f)) : 0.f;
                dyh = on ? dyh * (zf * sg) : 0.f;
            }
            if (step < L) {
                sdt[e] = dt;
                sdtu[e] = dt * uf[i];
                sdy[e] = dyh;
            }
        }
        stage_vecs<T, Gm>(sB, rB, lane);
        stage_vecs<T, Gm>(sC, rC, lane);
        __syncwarp();
        if (seg - kScanWarps >= 0) fetch(seg - kScanWarps);

        // forward through the segment: states, running decay, and the
        // segment's own part of the outgoing gradient
        f2 h[L][CH][2], p[CH][2], E[CH][2];
#pragma unroll
        for (int t = 0; t < L; ++t) {
            f2 B[2], C[2];
            lds_quad(B, sB + t * NP + 4 * nl);
            lds_quad(C, sC + t * NP + 4 * nl);
            float dt[CH], dtu[CH], dyh[CH];
            lds_run<CH>(dt, sdt + t * CPW + cl * CH);
            lds_run<CH>(dtu, sdtu + t * CPW + cl * CH);
            lds_run<CH>(dyh, sdy + t * CPW + cl * CH);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const f2 dt2 = pack2(dt[c], dt[c]), dtu2 = pack2(dtu[c], dtu[c]), dy2 = pack2(dyh[c], dyh[c]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 dec = ex2_pair(mul2(dt2, A[c][k]));
                    h[t][c][k] = fma2(dec, t == 0 ? h0[c][k] : h[t - 1][c][k], mul2(dtu2, B[k]));
                    p[c][k] = t == 0 ? dec : mul2(p[c][k], dec);
                    const f2 cd = mul2(C[k], dy2);
                    E[c][k] = t == 0 ? mul2(p[c][k], cd) : fma2(p[c][k], cd, E[c][k]);
                }
            }
        }
        // the gradient that reaches the segment's last state from later ones
        f2 g[CH][2];
        if (seg == nseg - 1) {
            if (a.dh_T) load_states<Gm>(g, a.dh_T + sbase, tl, a.N, a.state_vec, cl, nl, 1.f, false);
            else
#pragma unroll
                for (int c = 0; c < CH; ++c) g[c][0] = g[c][1] = pack2(0.f, 0.f);
        } else {
            carry_wait(warp);
#pragma unroll
            for (int c = 0; c < CH; ++c) lds_quad(g[c], carry + warp * Gm::QUADS + (c * 32 + lane) * 4);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k) E[c][k] = fma2(p[c][k], g[c][k], E[c][k]);
        if (seg > 0) {
            const int to = (warp + 1) % kScanWarps;
#pragma unroll
            for (int c = 0; c < CH; ++c) sts_quad(carry + to * Gm::QUADS + (c * 32 + lane) * 4, E[c]);
            carry_arrive(to);
        } else if (a.dh0) {
            store_states<Gm>(a.dh0 + sbase, E, tl, a.N, a.state_vec, cl, nl);
        }
        // back through the segment
#pragma unroll
        for (int t = L - 1; t >= 0; --t) {
            f2 B[2], C[2], dB[2], dC[2];
            lds_quad(B, sB + t * NP + 4 * nl);
            lds_quad(C, sC + t * NP + 4 * nl);
            float dt[CH], dtu[CH], dyh[CH], v[3 * CH];
            lds_run<CH>(dt, sdt + t * CPW + cl * CH);
            lds_run<CH>(dtu, sdtu + t * CPW + cl * CH);
            lds_run<CH>(dyh, sdy + t * CPW + cl * CH);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const f2 dt2 = pack2(dt[c], dt[c]), dtu2 = pack2(dtu[c], dtu[c]), dy2 = pack2(dyh[c], dyh[c]);
                f2 yc, gB, dd;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 dec = ex2_pair(mul2(dt2, A[c][k]));
                    const f2 gt = fma2(C[k], dy2, g[c][k]), ht = h[t][c][k];
                    yc = k == 0 ? mul2(C[k], ht) : fma2(C[k], ht, yc);
                    gB = k == 0 ? mul2(B[k], gt) : fma2(B[k], gt, gB);
                    dB[k] = c == 0 ? mul2(gt, dtu2) : fma2(gt, dtu2, dB[k]);
                    dC[k] = c == 0 ? mul2(ht, dy2) : fma2(ht, dy2, dC[k]);
                    g[c][k] = mul2(dec, gt);
                    const f2 w = mul2(g[c][k], t == 0 ? h0[c][k] : h[t - 1][c][k]);
                    dA[c][k] = fma2(w, dt2, dA[c][k]);
                    dd = k == 0 ? mul2(A[c][k], w) : fma2(A[c][k], w, dd);  // A log2(e) here
                }
                v[3 * c] = sum2(yc);
                v[3 * c + 1] = sum2(gB);
                v[3 * c + 2] = sum2(dd);
            }
            // over the states: values 3 c + {y, gB, dd}
            using Sum = LaneSum<3 * CH, NS, 1>;
            Sum::run(v, nl);
            if (Sum::owner(nl)) {
#pragma unroll
                for (int i = 0; i < Sum::left(); i += 3) {
                    const int at = t * CPW + cl * CH + (Sum::first(nl) + i) / 3;
                    sY[at] = v[i];
                    sGB[at] = v[i + 1];
                    sDD[at] = v[i + 2] * kLn2;
                }
            }
            // over the warp's channels: 4 states of dB, then of dC
            float w[8];
            unpack2(dB[0], w[0], w[1]);
            unpack2(dB[1], w[2], w[3]);
            unpack2(dC[0], w[4], w[5]);
            unpack2(dC[1], w[6], w[7]);
            using Bc = LaneSum<8, Gm::CL, NS>;
            Bc::run(w, lane);
            const int tok = seg * L + t;
            if (tok < tl.n && Bc::owner(lane)) {
                float* o = bcp + (size_t)tok * a.G * (2 * NP);
#pragma unroll
                for (int i = 0; i < Bc::left(); ++i) {
                    const int e = Bc::first(lane) + i;
                    o[(e >> 2) * NP + 4 * nl + (e & 3)] = w[i];
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < Gm::SE; ++i) {
            const int e = 32 * i + lane, step = e / CPW, ch = e % CPW, t = seg * L + step;
            if (step >= L || t >= a.T || ch >= tl.kleft) continue;
            const float dyh = sdy[e], gB = sGB[e];
            const bool on = t < tl.n;
            const float dd = on ? fmaf(uf[i], gB, sDD[e]) * sig[i] : 0.f;
            const size_t o = rbase + (size_t)t * a.D_ + ch;
            a.du[o] = on ? fmaf(sdt[e], gB, skip[i % AC] * dyh) : 0.f;
            a.ddelta[o] = dd;
            if (z) a.dz[o] = on ? gz[i] * fmaf(skip[i % AC], uf[i], sY[e]) : 0.f;
            dD[i % AC] = fmaf(dyh, uf[i], dD[i % AC]);
            db[i % AC] += dd;
        }
        __syncwarp();
    }
    // rows that hold no token
    for (int e = threadIdx.x; e < (a.T - min(a.T, nseg * L)) * CPW; e += kScanThreads) {
        const int t = nseg * L + e / CPW, ch = e % CPW;
        if (ch >= tl.kleft) continue;
        const size_t o = rbase + (size_t)t * a.D_ + ch;
        a.du[o] = a.ddelta[o] = 0.f;
        if (z) a.dz[o] = 0.f;
    }
    if (nseg == 0 && warp == 0 && a.dh0) {
        f2 g[CH][2];
        if (a.dh_T) load_states<Gm>(g, a.dh_T + sbase, tl, a.N, a.state_vec, cl, nl, 1.f, false);
        else
#pragma unroll
            for (int c = 0; c < CH; ++c) g[c][0] = g[c][1] = pack2(0.f, 0.f);
        store_states<Gm>(a.dh0 + sbase, g, tl, a.N, a.state_vec, cl, nl);
    }
    // the sequence's parameter gradients: warps added in order
    __syncthreads();
    float* red = sm;  // [warp][QUADS + 2 CPW]
    constexpr int kRed = Gm::QUADS + 2 * CPW;
#pragma unroll
    for (int c = 0; c < CH; ++c) sts_quad(red + warp * kRed + (c * 32 + lane) * 4, dA[c]);
#pragma unroll
    for (int i = 0; i < AC; ++i) {
#pragma unroll
        for (int m = CPW; m < 32; m <<= 1) {
            dD[i] += __shfl_xor_sync(0xffffffffu, dD[i], m);
            db[i] += __shfl_xor_sync(0xffffffffu, db[i], m);
        }
        if (lane < CPW) {
            red[warp * kRed + Gm::QUADS + 32 * i + lane] = dD[i];
            red[warp * kRed + Gm::QUADS + CPW + 32 * i + lane] = db[i];
        }
    }
    __syncthreads();
    float* prm = a.prm + (size_t)tl.b * a.D_ * (a.N + 2);
    for (int e = threadIdx.x; e < kRed; e += kScanThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) s += red[w * kRed + e];
        if (e < Gm::QUADS) {
            const int ln = (e >> 2) & 31, ch = (ln / NS) * CH + (e >> 7), n = (ln % NS) * 4 + (e & 3);
            if (ch < tl.kleft && n < a.N) prm[(size_t)(tl.c0 + ch) * a.N + n] = s;
        } else {
            const int r = e - Gm::QUADS, ch = r % CPW;
            if (ch < tl.kleft) prm[(size_t)a.D_ * (a.N + r / CPW) + tl.c0 + ch] = s;
        }
    }
}

// Adds the channel tiles of dB, dC (first `bc_blocks` blocks) and the
// sequences of dA, dD, ddelta_bias (the rest), each in order.
struct ScanReduce {
    const float *bcpart, *prm;
    const int* lengths;
    float *dB, *dC, *dA, *dD, *dbias;
    long long vecs;  // B * T * G
    int B, T, G, D_, N, NP, tiles;
    unsigned bc_blocks;
};

__global__ void __launch_bounds__(256) scan_reduce_kernel(ScanReduce r) {
    dependent_wait();
    if (blockIdx.x < r.bc_blocks) {
        const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
        const long long vec = e / (2 * r.NP);
        const int i = (int)(e - vec * (2 * r.NP)), n = i % r.NP;
        if (vec >= r.vecs || n >= r.N) return;
        const long long tok = vec / r.G;
        const int b = (int)(tok / r.T), t = (int)(tok - (long long)b * r.T);
        float s = 0.f;
        if (t < seq_len(r.lengths, b, r.T))
            for (int k = 0; k < r.tiles; ++k) s += r.bcpart[(size_t)k * r.vecs * (2 * r.NP) + e];
        (i < r.NP ? r.dB : r.dC)[vec * r.N + n] = s;
        return;
    }
    const long long e = (long long)(blockIdx.x - r.bc_blocks) * 256 + threadIdx.x;
    const long long da = (long long)r.D_ * r.N, all = da + 2ll * r.D_;
    if (e >= all) return;
    float s = 0.f;
    for (int b = 0; b < r.B; ++b) s += r.prm[(size_t)b * all + e];
    if (e < da) r.dA[e] = s;
    else if (e < da + r.D_) { if (r.dD) r.dD[e - da] = s; }
    else if (r.dbias) r.dbias[e - da - r.D_] = s;
}

cudaError_t launch_scan_ckpt(const ScanArgs& a, int B, int dtype, cudaStream_t st);

// Channels per tile of the backward geometry (2 per lane).
static int bwd_tiles(int K, int N) { const int cpw = 64 / scan_lanes(N); return (K + cpw - 1) / cpw; }
constexpr int kBwdL = 8;

struct ScanBwdLayout { size_t ckpt, bc, prm, total; };
ScanBwdLayout scan_bwd_layout(int B, int T, int D, int N, int G) {
    const size_t tiles = bwd_tiles(D / G, N), np = 4 * scan_lanes(N);
    ScanBwdLayout l;
    l.ckpt = 0;
    l.bc = l.ckpt + round256((size_t)B * G * tiles * ((T + kBwdL - 1) / kBwdL) * (2 * 32 * 4) * sizeof(float));
    l.prm = l.bc + round256(tiles * B * T * G * 2 * np * sizeof(float));
    l.total = l.prm + round256((size_t)B * D * (N + 2) * sizeof(float));
    return l;
}

template <typename T, typename TG, int NS> static cudaError_t launch_bwd_geom(ScanArgs a, int B, cudaStream_t st) {
    using Gm = ScanGeom<NS, 2, kBwdL>;
    constexpr size_t kRun = kScanWarps * (6 * Gm::L * Gm::CPW + 2 * Gm::L * Gm::NP + Gm::QUADS) * sizeof(float);
    constexpr size_t kRed = kScanWarps * (Gm::QUADS + 2 * Gm::CPW) * sizeof(float);
    constexpr size_t smem = kRun > kRed ? kRun : kRed;
    auto kern = scan_bwd_kernel<T, TG, Gm>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<(unsigned)((long long)B * a.G * a.tiles), kScanThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename TG> static cudaError_t launch_bwd_lanes(const ScanArgs& a, int B, cudaStream_t st) {
    switch (scan_lanes(a.N)) {
        case 1: return launch_bwd_geom<T, TG, 1>(a, B, st);
        case 2: return launch_bwd_geom<T, TG, 2>(a, B, st);
        case 4: return launch_bwd_geom<T, TG, 4>(a, B, st);
        case 8: return launch_bwd_geom<T, TG, 8>(a, B, st);
        case 16: return launch_bwd_geom<T, TG, 16>(a, B, st);
        default: return launch_bwd_geom<T, TG, 32>(a, B, st);
    }
}

cudaError_t launch_scan_bwd(ScanArgs a, void* ws, float* dA, float* dB, float* dC, float* dD, float* dbias, int B,
                            int dtype, int grad_dtype, cudaStream_t st) {
    const ScanBwdLayout l = scan_bwd_layout(B, a.T, a.D_, a.N, a.G);
    char* w = reinterpret_cast<char*>(ws);
    a.ckpt = reinterpret_cast<float*>(w + l.ckpt);
    a.bcpart = reinterpret_cast<float*>(w + l.bc);
    a.prm = reinterpret_cast<float*>(w + l.prm);
    a.nseg = (a.T + kBwdL - 1) / kBwdL;
    a.tiles = bwd_tiles(a.K, a.N);
    if ((long long)B * a.G * a.tiles > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaError_t e = a.T > 0 ? launch_scan_ckpt(a, B, dtype, st) : cudaSuccess;
    if (e != cudaSuccess) return e;
    e = dtype == GDR_FP32 ? launch_bwd_lanes<float, float>(a, B, st)
        : grad_dtype == GDR_FP32 ? launch_bwd_lanes<__nv_bfloat16, float>(a, B, st)
                                 : launch_bwd_lanes<__nv_bfloat16, __nv_bfloat16>(a, B, st);
    if (e != cudaSuccess) return e;
    ScanReduce r = {};
    r.bcpart = a.bcpart; r.prm = a.prm; r.lengths = a.lengths;
    r.dB = dB; r.dC = dC; r.dA = dA; r.dD = dD; r.dbias = dbias;
    r.vecs = (long long)B * a.T * a.G;
    r.B = B; r.T = a.T; r.G = a.G; r.D_ = a.D_; r.N = a.N; r.NP = 4 * scan_lanes(a.N); r.tiles = a.tiles;
    const long long bc = (r.vecs * 2 * r.NP + 255) / 256, pr = ((long long)a.D_ * (a.N + 2) + 255) / 256;
    if (bc + pr > 0x7fffffffll) return cudaErrorInvalidValue;
    r.bc_blocks = (unsigned)bc;
    return launch_dependent(scan_reduce_kernel, (unsigned)(bc + pr), 256, 0, st, r);
}

}  // namespace gdr
