// Selective state-space scan: backward pass.
//
// With g_t = dL/dh_t, yh = y before the gate and dyh = dy z sigmoid(z):
//   g_t = C_t dyh_t + a_{t+1} g_{t+1},  a = exp(dt A);   dh0 = a_1 g_1
//   dC_t = sum_d dyh h_t,  dB_t = sum_d dt u g_t
//   du = dt sum_n g B + D dyh,  d dt = sum_n g (u B + A a h_{t-1})
//   dA = sum dt a g h_{t-1},  dD = sum dyh u,  dz = dy yh (z sigmoid(z))'
//   ddelta = d dt sigmoid(delta + bias) (with softplus).
// Three launches. The forward scan first stores the state at the start of every
// segment of 8 tokens (scan.cu). The second walks the segments from the last to
// the first: a walker rebuilds a segment's states from the stored one, keeping
// states and decays in registers, and goes back through it. Sums over the states
// of a channel and over the channels of a block are left to the helpers, through
// shared memory. The third launch adds the blocks' dB and dC and the sequences'
// parameter gradients in a fixed order.
//
// Where the channels alone leave SMs empty the tokens are split into chunks, as
// in the forward pass: a launch before the others finds each chunk's maps of its
// start state (state -> P state + h) and of the gradient that reaches its end
// (gradient -> P gradient + E, E = sum_t p_t C_t dyh_t with the running decay p).
#include <type_traits>

#include "scan_common.cuh"

namespace gdr {

constexpr float kLn2 = 0.6931471805599453f;

template <typename T, typename TG, typename Gm> struct ScanBwdShared {
    static constexpr int L = Gm::Seg;
    // floats of a step: (dt, dt u) quads, dyh (twice where two blocks per SM leave
    // the room: a pair as the walkers need it), B, C
    static constexpr int kDup = sizeof(T) == 2 ? 2 : 1;
    static constexpr int dy = 4 * L * Gm::CB, B = dy + kDup * L * Gm::CB, in = B + 2 * L * Gm::NP;
    // of its results: sums of C h, g B and A a g h over the states, terms of dB and dC
    static constexpr int kSum = L * Gm::CB * Gm::NQ, bc = 3 * kSum, out = bc + L * 2 * kWalkers * 128;
    // of rows on their way: delta, u, z; dy; B and C
    using Rows = TokenRows<T, Gm, L>;
    using Grads = TokenRows<TG, Gm, L>;
    using States = StateRows<T, Gm, L>;
    static constexpr int slots = 3 * Rows::kWords + Grads::kWords + States::kWords;
    // and the state before each walker's next segment
    static constexpr int ckpt = 2 * (in + out + slots), total = ckpt + kWalkers * Gm::QUADS;
};

// ENDS: the chunk's maps only, its segments in order.
template <typename T, typename TG, typename Gm, bool ENDS>
__global__ void __launch_bounds__(kScanThreads, kBwdBlocks) scan_bwd_kernel(ScanArgs a) {
    constexpr int CH = Gm::CH, L = Gm::Seg, CB = Gm::CB, CL = Gm::CL, NP = Gm::NP, NS = Gm::NS, NQ = Gm::NQ;
    using Sh = ScanBwdShared<T, TG, Gm>;
    extern __shared__ __align__(16) float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ScanTile tl(a, CB);
    const int steps = (tl.n - tl.t0 + L - 1) / L;
    float* const results = sm + 2 * Sh::in;
    auto pair_at = [](const float* p, int at) {
        if constexpr (Sh::kDup == 2) return *reinterpret_cast<const f2*>(p + 2 * at);
        else return both2(p[at]);
    };
    auto segment = [&](int s) { return ENDS ? s : steps - 1 - s; };  // of step s
    float* const prm = a.prm + ((size_t)tl.b * a.chunks + tl.part) * a.D_ * (a.N + 2);

    if (warp < kWalkers) {
        const int nl = lane % NS, cl = lane / NS, at0 = lane_place<Gm>(warp, 0, cl);
        f2 A[CH][2];
        load_states<Gm, true>(A, a.A, tl, a.N, a.state_vec, at0, nl);
        if constexpr (ENDS) {
            f2 h[CH][2], p[CH][2], E[CH][2];
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    h[c][k] = E[c][k] = both2(0.f);
                    p[c][k] = both2(1.f);
                }
            __syncthreads();
            for (int s = 0; s <= steps; ++s) {
                const float* in = sm + (s & 1) * Sh::in;
                if (s < steps) {
#pragma unroll
                    for (int t = 0; t < L; ++t) {
                        f2 B[2], C[2];
                        lds_quad(B, in + Sh::B + t * NP + 4 * nl);
                        lds_quad(C, in + Sh::B + (L + t) * NP + 4 * nl);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const int at = t * CB + c * CL + at0;
                            f2 d[2];
                            lds_quad(d, in + at * 4);
                            const f2 dyh = pair_at(in + Sh::dy, at);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const f2 e = decay2(d[0], A[c][k]);
                                h[c][k] = fma2(e, h[c][k], mul2(d[1], B[k]));
                                p[c][k] = mul2(p[c][k], e);
                                E[c][k] = fma2(p[c][k], mul2(C[k], dyh), E[c][k]);
                            }
                        }
                    }
                }
                __syncthreads();
            }
            store_map<Gm>(a.ends, p, h, a, tl, warp, lane);
            store_map<Gm>(a.grad_ends, p, E, a, tl, warp, lane);
        } else {
            f2 dA[CH][2], g[CH][2];  // dA: a sum of the segments' sums, for accuracy
            load_given<Gm>(g, a.dh_T, a, tl, at0, nl);
            fold_chunks<Gm>(g, a.grad_ends, a, tl, warp, lane, a.chunks - 1, tl.part, -1);
#pragma unroll
            for (int c = 0; c < CH; ++c) dA[c][0] = dA[c][1] = both2(0.f);
            const float* ckpt = a.ckpt + ((tl.unit * kWalkers + warp) * a.segs + tl.t0 / L) * Gm::QUADS + lane * 4;
            float* const before = sm + Sh::ckpt + warp * Gm::QUADS + lane * 4;  // a lane's own quads
            auto fetch = [&](int s) {
                if (s < steps)
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        slot_fetch<float, 4>(reinterpret_cast<uint32_t*>(before + c * 128),
                                             ckpt + (size_t)segment(s) * Gm::QUADS + c * 128, true, 4, kWhole);
                copies_commit();
            };
            fetch(0);
            __syncthreads();
            for (int s = 0; s <= steps; ++s) {
                if (s < steps) {
                    const float* in = sm + (s & 1) * Sh::in;
                    float* o = results + (s & 1) * Sh::out;
                    f2 h0[CH][2], h[L][CH][2], dec[L][CH][2];
                    copies_wait<0>();
#pragma unroll
                    for (int c = 0; c < CH; ++c) lds_quad(h0[c], before + c * 128);
#pragma unroll
                    for (int t = 0; t < L; ++t) {
                        f2 B[2];
                        lds_quad(B, in + Sh::B + t * NP + 4 * nl);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            f2 d[2];
                            lds_quad(d, in + (t * CB + c * CL + at0) * 4);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                dec[t][c][k] = decay2(d[0], A[c][k]);
                                h[t][c][k] = fma2(dec[t][c][k], t == 0 ? h0[c][k] : h[t - 1][c][k], mul2(d[1], B[k]));
                            }
                        }
                    }
                    fetch(s + 1);  // h0 has been used
                    // a token's operands are loaded before the last one's sums are
                    // stored: the compiler cannot tell that the two do not overlap
                    struct { f2 B[2], C[2], d[CH][2], dyh[CH]; } x, next;  // d: dt, dt u
                    auto load = [&](decltype(x)& v, int t) {
                        lds_quad(v.B, in + Sh::B + t * NP + 4 * nl);
                        lds_quad(v.C, in + Sh::B + (L + t) * NP + 4 * nl);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const int at = t * CB + c * CL + at0;
                            lds_quad(v.d[c], in + at * 4);
                            v.dyh[c] = pair_at(in + Sh::dy, at);
                        }
                    };
                    load(x, L - 1);
                    f2 part[CH][2];
#pragma unroll
                    for (int t = L - 1; t >= 0; --t) {
                        if (t > 0) load(next, t - 1);
                        f2 dB[2], dC[2];
                        float vy[CH], vg[CH], vd[CH];
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            f2 yc, gB, dd;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const f2 gt = fma2(x.C[k], x.dyh[c], g[c][k]), ht = h[t][c][k];
                                yc = k == 0 ? mul2(x.C[k], ht) : fma2(x.C[k], ht, yc);
                                gB = k == 0 ? mul2(x.B[k], gt) : fma2(x.B[k], gt, gB);
                                dB[k] = c == 0 ? mul2(gt, x.d[c][1]) : fma2(gt, x.d[c][1], dB[k]);
                                dC[k] = c == 0 ? mul2(ht, x.dyh[c]) : fma2(ht, x.dyh[c], dC[k]);
                                g[c][k] = mul2(dec[t][c][k], gt);
                                const f2 w = mul2(g[c][k], t == 0 ? h0[c][k] : h[t - 1][c][k]);
                                part[c][k] = t == L - 1 ? mul2(w, x.d[c][0]) : fma2(w, x.d[c][0], part[c][k]);
                                dd = k == 0 ? mul2(A[c][k], w) : fma2(A[c][k], w, dd);  // A log2(e) here
                            }
                            vy[c] = fold_states<Gm>(sum2(yc));
                            vg[c] = fold_states<Gm>(sum2(gB));
                            vd[c] = fold_states<Gm>(sum2(dd));
                        }
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const int at = (t * CB + c * CL + at0) * NQ + nl;
                            if (nl < NQ) {
                                o[at] = vy[c];
                                o[Sh::kSum + at] = vg[c];
                                o[2 * Sh::kSum + at] = vd[c];
                            }
                        }
                        sts_quad(o + Sh::bc + ((2 * t) * kWalkers + warp) * 128 + lane * 4, dB);
                        sts_quad(o + Sh::bc + ((2 * t + 1) * kWalkers + warp) * 128 + lane * 4, dC);
                        x = next;
                    }
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int k = 0; k < 2; ++k) dA[c][k] = add2(dA[c][k], part[c][k]);
                }
                __syncthreads();
            }
            if (a.dh0 && tl.part == 0) store_states<Gm>(a.dh0, g, a, tl, at0, nl);
            // dA: this block's part, a lane's own states
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float f[4];
                unpack2(dA[c][0], f[0], f[1]);
                unpack2(dA[c][1], f[2], f[3]);
                const int ch = place_channel<Gm>(at0 + c * CL);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (ch < tl.kleft && nl * 4 + i < a.N) prm[(size_t)(tl.c0 + ch) * a.N + nl * 4 + i] = f[i];
            }
        }
    } else {
        const int ht = threadIdx.x - 32 * kWalkers;
        using Rows = typename Sh::Rows;
        constexpr int VW = Rows::VW;
        const int vch = Rows::channel(ht);
        const T* u = reinterpret_cast<const T*>(a.u) + tl.b * a.us[0] + tl.c0;
        const T* dl = reinterpret_cast<const T*>(a.delta) + tl.b * a.ds[0] + tl.c0;
        const T* z = a.z ? reinterpret_cast<const T*>(a.z) + tl.b * a.zs[0] + tl.c0 : nullptr;
        const TG* dy = reinterpret_cast<const TG*>(a.dy) + tl.b * a.gs[0] + tl.c0;
        const T* Bm = reinterpret_cast<const T*>(a.Bm) + tl.b * a.bs[0] + tl.g * a.N;
        const T* Cm = reinterpret_cast<const T*>(a.Cm) + tl.b * a.cs[0] + tl.g * a.N;
        const size_t rbase = (size_t)tl.b * a.T * a.D_ + tl.c0 + vch;
        float* bcp = a.bcpart + (((size_t)tl.tile * (gridDim.x / (a.tiles * a.chunks * a.G)) + tl.b) * a.T * a.G + tl.g) * (2 * NP);
        using Grads = typename Sh::Grads;
        using States = typename Sh::States;
        // what the output needs of the segments staged and walked: u, ddt/ddelta,
        // dy dgate/dz, dt, dyh
        struct Held { Rows u; float sig[Rows::NV][VW], gz[Rows::NV][VW], dt[Rows::NV][VW], dyh[Rows::NV][VW]; } held[2];
        uint32_t* const slots = reinterpret_cast<uint32_t*>(results + 2 * Sh::out);
        float bias[VW], skip[VW], dD[VW], lost[VW], db[VW];
#pragma unroll
        for (int j = 0; j < VW; ++j) dD[j] = lost[j] = db[j] = 0.f;
        channel_values(bias, a.bias, tl, vch);
        channel_values(skip, a.D, tl, vch);
        constexpr int kGrads = 3 * Rows::kWords, kStates = kGrads + Grads::kWords;
        auto fetch = [&](int s) {  // into the slots of step s - 2
            uint32_t* w = slots + (s & 1) * Sh::slots;
            if (s < steps) {
                const int t0 = tl.t0 + segment(s) * L;
                if (copies_fit<T>(a.act_vec)) {
                    Rows::fetch(w, dl, a.ds[1], t0, tl, a.act_vec, ht);
                    Rows::fetch(w + Rows::kWords, u, a.us[1], t0, tl, a.act_vec, ht);
                    if (z) Rows::fetch(w + 2 * Rows::kWords, z, a.zs[1], t0, tl, a.act_vec, ht);
                    Grads::fetch(w + kGrads, dy, a.gs[1], t0, tl, a.act_vec, ht);
                } else {
                    Rows r[3];
                    Grads g;
                    r[0].load(dl, a.ds[1], t0, tl, ht);
                    r[1].load(u, a.us[1], t0, tl, ht);
                    if (z) r[2].load(z, a.zs[1], t0, tl, ht);
                    g.load(dy, a.gs[1], t0, tl, ht);
                    r[0].store(w, ht);
                    r[1].store(w + Rows::kWords, ht);
                    if (z) r[2].store(w + 2 * Rows::kWords, ht);
                    g.store(w + kGrads, ht);
                }
                States::fetch(w + kStates, Bm, Cm, a, t0, tl, a.bc_vec, ht);
            }
            copies_commit();
        };
        // A step is one stretch of code without branches, so that the chains of the
        // rows coming in and of the sums going out fill each other's waits.
        Rows rd, rz;
        Grads rg;
        auto read = [&](int s) {
            const uint32_t* w = slots + (s & 1) * Sh::slots;
            held[0] = held[1];
            copies_wait<1>();
            rd.read(w, ht);
            held[1].u.read(w + Rows::kWords, ht);
            rz.read(w + 2 * Rows::kWords, ht);  // not used without z
            rg.read(w + kGrads, ht);
        };
        auto stage = [&](int s) {  // beyond the last step into a buffer that nobody reads
            float* in = sm + (s & 1) * Sh::in;
            const uint32_t* w = slots + (s & 1) * Sh::slots;
#pragma unroll
            for (int i = 0; i < Rows::NV; ++i) {
                const int tok = Rows::token(i, ht);
                const bool on = tl.t0 + segment(s) * L + tok < tl.n && vch < tl.kleft;
                float raw[VW], uf[VW], dt[VW], g[VW];
                raw_floats(raw, rd.v[i]);
                raw_floats(uf, held[1].u.v[i]);
                raw_floats(g, rg.v[i]);
#pragma unroll
                for (int j = 0; j < VW; ++j) raw[j] += bias[j];
                step_sizes<!ENDS>(dt, held[1].sig[i], raw, a.softplus);
#pragma unroll
                for (int j = 0; j < VW; j += 2) {
                    if (z) {
                        const f2 zz = pack2(rz.v[i].get(j), rz.v[i].get(j + 1)), sz = sigmoid2(zz),
                                 gg = pack2(g[j], g[j + 1]);
                        // (z s)' = s (1 + z (1 - s))
                        if (!ENDS)
                            unpack2(mul2(gg, mul2(sz, fma2(zz, fma2(sz, both2(-1.f), both2(1.f)), both2(1.f)))),
                                    held[1].gz[i][j], held[1].gz[i][j + 1]);
                        unpack2(mul2(gg, mul2(zz, sz)), g[j], g[j + 1]);
                    }
                }
                if (tok < L)
#pragma unroll
                    for (int j = 0; j < VW; ++j) {
                        const float d = on ? dt[j] : 0.f, gy = on ? g[j] : 0.f;
                        const f2 q[2] = {both2(d), both2(d * uf[j])};
                        const int at = tok * CB + channel_place<Gm>(vch + j);
                        held[1].dt[i][j] = d;
                        held[1].dyh[i][j] = gy;
                        sts_quad(in + at * 4, q);
                        if constexpr (Sh::kDup == 2) *reinterpret_cast<f2*>(in + Sh::dy + at * 2) = both2(gy);
                        else in[Sh::dy + at] = gy;
                    }
            }
            States::stage(w + kStates, in + Sh::B, ht, true);
        };
        auto put_out = [&](int s, const Held& h) {
            const float* o = results + (s & 1) * Sh::out;
            const int t0 = tl.t0 + segment(s) * L;
#pragma unroll
            for (int i = 0; i < Rows::NV; ++i) {
                const int tok = Rows::token(i, ht) % L, t = t0 + tok;  // % L: threads beyond the rows repeat some
                const bool live = Rows::token(i, ht) < L && t < tl.t1 && vch < tl.kleft, on = live && t < tl.n;
                float uf[VW], du[VW], dd[VW], dz[VW];
                raw_floats(uf, h.u.v[i]);
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const int at = tok * CB + channel_place<Gm>(vch + j);
                    const float dt = h.dt[i][j], dyh = h.dyh[i][j];
                    const float gB = sum_states<Gm>(o + Sh::kSum + at * NQ);
                    const float sd = sum_states<Gm>(o + 2 * Sh::kSum + at * NQ) * kLn2;
                    du[j] = fmaf(dt, gB, skip[j] * dyh);
                    dd[j] = fmaf(uf[j], gB, sd) * h.sig[i][j];
                    dz[j] = z ? h.gz[i][j] * fmaf(skip[j], uf[j], sum_states<Gm>(o + at * NQ)) : 0.f;
                    if (!on) du[j] = dd[j] = dz[j] = 0.f;
                    // a thread adds hundreds of tokens: what an addition loses goes into the
                    // next one (without that dD is 3.9e-7 off, with it 0.9e-7)
                    const float term = on ? fmaf(dyh, uf[j], -lost[j]) : -lost[j], sum = dD[j] + term;
                    // finite (NaN gives the bound), so that an infinite sum stays infinite
                    lost[j] = fminf(fmaxf((sum - dD[j]) - term, -1e36f), 1e36f);
                    dD[j] = sum;
                    db[j] += dd[j];
                }
                const size_t row = rbase + (size_t)t * a.D_;
                if (live) {
                    store_row(a.du + row, du, tl.kleft - vch, a.out_vec);
                    store_row(a.ddelta + row, dd, tl.kleft - vch, a.out_vec);
                    if (z) store_row(a.dz + row, dz, tl.kleft - vch, a.out_vec);
                }
            }
            // dB, dC over the block's channels: quad e is token e / (2 NS), B or C, 4
            // states; F threads add up to 4 CL terms, each row from another lane on
            // (for the banks)
            // (threads of a quad start a lane apart too, where each has whole rows)
            constexpr int Q = L * 2 * NS, F = Q < kHelperThreads ? kHelperThreads / Q : 1, kTerms = kWalkers * CL / F;
#pragma unroll
            for (int q0 = 0; q0 < Q; q0 += kHelperThreads / F) {
                const int e = q0 + ht / F, row = e / NS, first = ht % F * kTerms, t = t0 + row / 2;
                const int turn = row + (kTerms % CL ? 0 : ht % F);
                f2 v[2] = {both2(0.f), both2(0.f)};
#pragma unroll
                for (int k = 0; k < kTerms; ++k) {
                    const int term = first + k;
                    f2 x[2];
                    lds_quad(x, o + Sh::bc + (row * kWalkers + term / CL) * 128 + ((term + turn) % CL * NS + e % NS) * 4);
                    v[0] = add2(v[0], x[0]);
                    v[1] = add2(v[1], x[1]);
                }
#pragma unroll
                for (int m = 1; m < F; m <<= 1) {
                    v[0] = add2(v[0], __shfl_xor_sync(0xffffffffu, v[0], m));
                    v[1] = add2(v[1], __shfl_xor_sync(0xffffffffu, v[1], m));
                }
                if (ht % F == 0 && t < tl.n) sts_quad(bcp + (size_t)t * a.G * (2 * NP) + (row & 1) * NP + e % NS * 4, v);
            }
        };
        auto bring_in = [&](int s) {
            read(s);
            stage(s);
            fetch(s + 2);
        };
        fetch(0);
        fetch(1);
        bring_in(0);
        __syncthreads();
        bring_in(1);
        __syncthreads();
        for (int s = 1; s <= steps; ++s) {
            const Held last = held[0];
            read(s + 1);
            if (!ENDS) put_out(s - 1, last);
            stage(s + 1);
            fetch(s + 2 + 1);
            __syncthreads();
        }
        if constexpr (!ENDS) {
            // rows that hold no token
            const int t0 = min(tl.t1, tl.t0 + steps * L);
            for (int e = ht; e < (tl.t1 - t0) * CB; e += kHelperThreads) {
                if (e % CB >= tl.kleft) continue;
                const size_t o = rbase - vch + (size_t)(t0 + e / CB) * a.D_ + e % CB;
                a.du[o] = a.ddelta[o] = 0.f;
                if (z) a.dz[o] = 0.f;
            }
            // dD, ddelta_bias: threads of a channel added in order
            constexpr int kShare = kHelperThreads / Rows::VPT;
            float* red = sm;  // [dD, db][share][CB]
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                red[ht / Rows::VPT * CB + vch + j] = dD[j];
                red[(kShare + ht / Rows::VPT) * CB + vch + j] = db[j];
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kHelperThreads) : "memory");
            for (int e = ht; e < 2 * CB; e += kHelperThreads) {
                const int which = e / CB, ch = e % CB;
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < kShare; ++k) v += red[(which * kShare + k) * CB + ch];
                if (ch < tl.kleft) prm[(size_t)a.D_ * (a.N + which) + tl.c0 + ch] = v;
            }
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
    int T, G, D_, N, NP, tiles, parts, wide;  // parts: sequences x chunks; wide: 16-byte stores
    unsigned bc_blocks;
};

__global__ void __launch_bounds__(256) scan_reduce_kernel(ScanReduce r) {
    dependent_wait();
    if (blockIdx.x < r.bc_blocks) {
        // 4 states of one token's dB or dC per thread, eight tiles on their way
        const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
        const int quads = r.NP / 2;  // of a token's B and C
        const long long vec = e / quads;
        const int i = (int)(e - vec * quads) * 4, n = i % r.NP;
        if (vec >= r.vecs || n >= r.N) return;
        const long long tok = vec / r.G;
        const int b = (int)(tok / r.T), t = (int)(tok - (long long)b * r.T);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const float4* p = reinterpret_cast<const float4*>(r.bcpart) + e;
        const size_t stride = (size_t)r.vecs * quads;
        if (t < seq_len(r.lengths, b, r.T)) {
#pragma unroll 8
            for (int k = 0; k < r.tiles; ++k) {
                const float4 v = p[k * stride];
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            }
        }
        float* o = (i < r.NP ? r.dB : r.dC) + vec * r.N + n;
        if (r.wide) VecIO<float, 4>::store(o, s);
        else
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < r.N) o[j] = s[j];
        return;
    }
    const long long e = (long long)(blockIdx.x - r.bc_blocks) * 256 + threadIdx.x;
    const long long da = (long long)r.D_ * r.N, all = da + 2ll * r.D_;
    if (e >= all) return;
    double sum = 0.;  // of some 300 chunks at most, or of any number of sequences
#pragma unroll 8
    for (int b = 0; b < r.parts; ++b) sum += r.prm[(size_t)b * all + e];
    const float s = (float)sum;
    if (e < da) r.dA[e] = s;
    else if (e < da + r.D_) { if (r.dD) r.dD[e - da] = s; }
    else if (r.dbias) r.dbias[e - da - r.D_] = s;
}

cudaError_t launch_scan_ckpt(const ScanArgs& a, int B, int dtype, cudaStream_t st);
void scan_split(ScanArgs& a, int chunks, int CH);
size_t scan_ends_bytes(int B, int G, int K, int N, int chunks, int CH);

// Chunks of the backward pass: the maps cost a third walk beside two, so two chunks
// pay already. One sequence of 2048 channels x 16 states in bf16: 384 tokens 79.5 us
// whole, 512 78.3 in two chunks. The 256 tokens at least are not borne out for short
// sequences: with 64, 384 would take 52.4 us and 512 63.2; from 1024 on nothing changes.
int scan_bwd_chunks(int B, int T, int K, int N, int G) {
    const long long units = (long long)B * G * scan_tiles(K, N, 1);
    const long long c = units > 0 ? 148 * kBwdBlocks / units : 0, most = T / 256;
    const long long n = c < most ? c : most;
    return n < 2 ? 1 : (int)n;
}

static int bwd_segments(int T, int N) { const int l = scan_segment(scan_lanes(N)); return (T + l - 1) / l; }

struct ScanBwdLayout { size_t ckpt, bc, prm, ends, grad_ends, total; };
ScanBwdLayout scan_bwd_layout(int B, int T, int D, int N, int G, int chunks) {
    const size_t tiles = scan_tiles(D / G, N, 1), np = 4 * scan_lanes(N), ends = scan_ends_bytes(B, G, D / G, N, chunks, 1);
    ScanBwdLayout l;
    l.ckpt = 0;
    l.bc = l.ckpt + round256((size_t)B * G * tiles * kWalkers * bwd_segments(T, N) * ScanBwdGeom<1>::QUADS * sizeof(float));
    l.prm = l.bc + round256(tiles * B * T * G * 2 * np * sizeof(float));
    l.ends = l.prm + round256((size_t)B * chunks * D * (N + 2) * sizeof(float));
    l.grad_ends = l.ends + ends;
    l.total = l.grad_ends + ends;
    return l;
}

template <typename T, typename TG, int NS, bool ENDS>
static cudaError_t launch_bwd_geom(const ScanArgs& a, int B, cudaStream_t st) {
    using Gm = ScanBwdGeom<NS>;
    constexpr size_t smem = ScanBwdShared<T, TG, Gm>::total * sizeof(float);
    static_assert(smem <= 227 * 1024, "shared memory of a block");
    auto kern = scan_bwd_kernel<T, TG, Gm, ENDS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)B * a.G * a.tiles * a.chunks), kScanThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename TG, bool ENDS> static cudaError_t launch_bwd_lanes(const ScanArgs& a, int B, cudaStream_t st) {
    switch (scan_lanes(a.N)) {
        case 1: return launch_bwd_geom<T, TG, 1, ENDS>(a, B, st);
        case 2: return launch_bwd_geom<T, TG, 2, ENDS>(a, B, st);
        case 4: return launch_bwd_geom<T, TG, 4, ENDS>(a, B, st);
        case 8: return launch_bwd_geom<T, TG, 8, ENDS>(a, B, st);
        case 16: return launch_bwd_geom<T, TG, 16, ENDS>(a, B, st);
        default: return launch_bwd_geom<T, TG, 32, ENDS>(a, B, st);
    }
}
template <bool ENDS>
static cudaError_t launch_bwd_types(const ScanArgs& a, int B, int dtype, int grad_dtype, cudaStream_t st) {
    return dtype == GDR_FP32        ? launch_bwd_lanes<float, float, ENDS>(a, B, st)
           : grad_dtype == GDR_FP32 ? launch_bwd_lanes<__nv_bfloat16, float, ENDS>(a, B, st)
                                    : launch_bwd_lanes<__nv_bfloat16, __nv_bfloat16, ENDS>(a, B, st);
}

cudaError_t launch_scan_bwd(ScanArgs a, void* ws, float* dA, float* dB, float* dC, float* dD, float* dbias, int B,
                            int dtype, int grad_dtype, cudaStream_t st) {
    const int chunks = scan_bwd_chunks(B, a.T, a.K, a.N, a.G);
    const ScanBwdLayout l = scan_bwd_layout(B, a.T, a.D_, a.N, a.G, chunks);
    char* w = reinterpret_cast<char*>(ws);
    a.ckpt = reinterpret_cast<float*>(w + l.ckpt);
    a.bcpart = reinterpret_cast<float*>(w + l.bc);
    a.prm = reinterpret_cast<float*>(w + l.prm);
    a.ends = reinterpret_cast<float*>(w + l.ends);
    a.grad_ends = reinterpret_cast<float*>(w + l.grad_ends);
    a.segs = bwd_segments(a.T, a.N);
    scan_split(a, chunks, 1);
    if ((long long)B * a.G * a.tiles * a.chunks > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaError_t e = a.chunks > 1 ? launch_bwd_types<true>(a, B, dtype, grad_dtype, st) : cudaSuccess;
    if (e != cudaSuccess) return e;
    e = a.T > 0 ? launch_scan_ckpt(a, B, dtype, st) : cudaSuccess;
    if (e != cudaSuccess) return e;
    e = launch_bwd_types<false>(a, B, dtype, grad_dtype, st);
    if (e != cudaSuccess) return e;
    ScanReduce r = {};
    r.bcpart = a.bcpart; r.prm = a.prm; r.lengths = a.lengths;
    r.dB = dB; r.dC = dC; r.dA = dA; r.dD = dD; r.dbias = dbias;
    r.vecs = (long long)B * a.T * a.G;
    r.T = a.T; r.G = a.G; r.D_ = a.D_; r.N = a.N; r.NP = 4 * scan_lanes(a.N); r.tiles = a.tiles;
    r.parts = B * a.chunks;
    r.wide = a.N % 4 == 0 && aligned_to(dB, 16) && aligned_to(dC, 16);
    const long long bc = (r.vecs * (r.NP / 2) + 255) / 256, pr = ((long long)a.D_ * (a.N + 2) + 255) / 256;
    if (bc + pr > 0x7fffffffll) return cudaErrorInvalidValue;
    r.bc_blocks = (unsigned)bc;
    return launch_dependent(scan_reduce_kernel, (unsigned)(bc + pr), 256, 0, st, r);
}

}  // namespace gdr
