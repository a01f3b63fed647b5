// Entry points of the selective state-space scan (include/gdr.h): argument
// checks on the host and the kernels' argument block.
#include "scan_common.cuh"

namespace gdr {
cudaError_t launch_scan_fwd(const ScanArgs& a, int B, int dtype, cudaStream_t st);
cudaError_t launch_scan_step(ScanArgs a, float* h, int B, int dtype, cudaStream_t st);
cudaError_t launch_scan_bwd(ScanArgs a, void* ws, float* dA, float* dB, float* dC, float* dD, float* dbias, int B,
                            int dtype, int grad_dtype, cudaStream_t st);
struct ScanBwdLayout { size_t ckpt, bc, prm, ends, grad_ends, total; };
ScanBwdLayout scan_bwd_layout(int B, int T, int D, int N, int G, int chunks);
int scan_chunks(int B, int T, int K, int N, int G);
int scan_bwd_chunks(int B, int T, int K, int N, int G);
void scan_split(ScanArgs& a, int chunks, int CH);
size_t scan_ends_bytes(int B, int G, int K, int N, int chunks, int CH);
}  // namespace gdr

using namespace gdr;

// Checks what every call has and fills the block; `strides` holds the batch
// and token strides of u, delta, Bm, Cm, z (and dy), or is null for dense arrays.
static gdr_status scan_fill(ScanArgs& a, const void* u, const void* delta, const float* A, const void* Bm,
                            const void* Cm, const float* D, const void* z, const float* delta_bias, const float* h0,
                            const int* lengths, const long long* strides, bool with_dy, int B, int T, int D_, int N,
                            int G, int delta_softplus, int dtype) {
    if (B < 1 || T < 0 || D_ < 1 || N < 1 || G < 1 || D_ % G || !dtype_ok(dtype)) return GDR_ERR_INVALID_ARG;
    if (!A || (T > 0 && (!u || !delta || !Bm || !Cm))) return GDR_ERR_INVALID_ARG;
    if (N > 128 || !axes_fit({B, T, D_})) return GDR_ERR_UNSUPPORTED;
    const size_t e = dtype_size(dtype);
    for (const void* p : {u, delta, Bm, Cm, z})
        if (!aligned_to(p, e)) return GDR_ERR_MISALIGNED;
    for (const void* p : {(const void*)A, (const void*)D, (const void*)delta_bias, (const void*)h0,
                          (const void*)lengths})
        if (!aligned_to(p, 4)) return GDR_ERR_MISALIGNED;
    a = ScanArgs{};
    a.u = u; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.z = z;
    a.bias = delta_bias; a.h0 = h0; a.lengths = lengths;
    a.T = T; a.D_ = D_; a.N = N; a.G = G; a.K = D_ / G; a.softplus = delta_softplus != 0;
    const long long td = (long long)T * D_, tn = (long long)T * G * N, gn = (long long)G * N;
    const long long dense[12] = {td, D_, td, D_, tn, gn, tn, gn, td, D_, td, D_};
    const long long* s = strides ? strides : dense;
    for (int i = 0; i < 2; ++i) {
        a.us[i] = s[i]; a.ds[i] = s[2 + i]; a.bs[i] = s[4 + i]; a.cs[i] = s[6 + i]; a.zs[i] = s[8 + i];
        if (with_dy) a.gs[i] = s[10 + i];
    }
    // B and C, and the token rows, in aligned vectors of 4 or pairs (dy: see gdr_scan_bwd)
    auto bc = [&](int m) {
        bool ok = N % m == 0 && aligned_to(Bm, m * e) && aligned_to(Cm, m * e);
        for (int i = 0; i < 2; ++i) ok = ok && a.bs[i] % m == 0 && a.cs[i] % m == 0;
        return ok;
    };
    auto rows = [&](int m) {
        bool ok = a.K % m == 0 && aligned_to(u, m * e) && aligned_to(delta, m * e) && aligned_to(z, m * e);
        for (int i = 0; i < 2; ++i)
            ok = ok && a.us[i] % m == 0 && a.ds[i] % m == 0 && (!z || a.zs[i] % m == 0) && a.gs[i] % m == 0;
        return ok;
    };
    a.bc_vec = bc(4) ? kWhole : bc(2) ? kPairs : kSingle;
    a.act_vec = rows(4) ? kWhole : rows(2) ? kPairs : kSingle;
    return GDR_OK;
}

// State arrays in 16-byte pieces: whole quads per channel and aligned arrays.
static int states_in_quads(int N, std::initializer_list<const void*> ptrs) {
    if (N % 4) return 0;
    for (const void* p : ptrs)
        if (!aligned_to(p, 16)) return 0;
    return 1;
}

static gdr_status launched(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH; }

extern "C" {

size_t gdr_scan_fwd_workspace_size(int B, int T, int D_, int N, int G) {
    if (B < 1 || T < 0 || D_ < 1 || N < 1 || N > 128 || G < 1 || D_ % G || !axes_fit({B, T, D_})) return 0;
    return scan_ends_bytes(B, G, D_ / G, N, scan_chunks(B, T, D_ / G, N, G), 2);
}

gdr_status gdr_scan_fwd(const void* u, const void* delta, const float* A, const void* Bm, const void* Cm,
                        const float* D, const void* z, const float* delta_bias, const float* h0, const int* lengths,
                        void* y, float* h_T, void* workspace, size_t workspace_bytes, const long long* strides, int B, int T, int D_, int N, int G,
                        int delta_softplus, int dtype, void* stream) {
    ScanArgs a;
    gdr_status ok = scan_fill(a, u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, strides, false, B, T, D_, N, G,
                              delta_softplus, dtype);
    if (ok != GDR_OK) return ok;
    if (T > 0 && !y) return GDR_ERR_INVALID_ARG;
    if (!aligned_to(y, dtype_size(dtype)) || !aligned_to(h_T, 4)) return GDR_ERR_MISALIGNED;
    a.y = y; a.h_T = h_T;
    a.out_vec = a.K % 4 == 0 && aligned_to(y, 4 * dtype_size(dtype));
    a.state_vec = states_in_quads(N, {A, h0, h_T});
    if (workspace && !aligned_to(workspace, 256)) return GDR_ERR_MISALIGNED;
    const size_t need = gdr_scan_fwd_workspace_size(B, T, D_, N, G);
    const bool split = workspace && need && workspace_bytes >= need;
    a.ends = reinterpret_cast<float*>(workspace);
    scan_split(a, split ? scan_chunks(B, T, a.K, N, G) : 1, 2);
    return launched(launch_scan_fwd(a, B, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdr_scan_bwd_workspace_size(int B, int T, int D_, int N, int G) {
    if (B < 1 || T < 0 || D_ < 1 || N < 1 || N > 128 || G < 1 || D_ % G || !axes_fit({B, T, D_})) return 0;
    return scan_bwd_layout(B, T, D_, N, G, scan_bwd_chunks(B, T, D_ / G, N, G)).total;
}

gdr_status gdr_scan_bwd(const void* u, const void* delta, const float* A, const void* Bm, const void* Cm,
                        const float* D, const void* z, const float* delta_bias, const float* h0, const int* lengths,
                        const void* dy, const float* dh_T, float* du, float* ddelta, float* dA, float* dB, float* dC,
                        float* dD, float* dz, float* ddelta_bias, float* dh0, void* workspace, size_t workspace_bytes,
                        const long long* strides, int B, int T, int D_, int N, int G, int delta_softplus, int dtype,
                        int grad_dtype, void* stream) {
    ScanArgs a;
    gdr_status ok = scan_fill(a, u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, strides, true, B, T, D_, N, G,
                              delta_softplus, dtype);
    if (ok != GDR_OK) return ok;
    if (!dtype_ok(grad_dtype)) return GDR_ERR_INVALID_ARG;
    if (grad_dtype != dtype && grad_dtype != GDR_FP32) return GDR_ERR_UNSUPPORTED;
    if (!dA || (T > 0 && (!dy || !du || !ddelta || !dB || !dC))) return GDR_ERR_INVALID_ARG;
    if ((dD != nullptr) != (D != nullptr) || (ddelta_bias != nullptr) != (delta_bias != nullptr) || (dh0 && !h0))
        return GDR_ERR_INVALID_ARG;
    if (T > 0 && (dz != nullptr) != (z != nullptr)) return GDR_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdr_scan_bwd_workspace_size(B, T, D_, N, G)) return GDR_ERR_INVALID_ARG;
    if (!aligned_to(workspace, 256) || !aligned_to(dy, dtype_size(grad_dtype))) return GDR_ERR_MISALIGNED;
    for (const void* p : {(const void*)dh_T, (const void*)du, (const void*)ddelta, (const void*)dA, (const void*)dB,
                          (const void*)dC, (const void*)dD, (const void*)dz, (const void*)ddelta_bias,
                          (const void*)dh0})
        if (!aligned_to(p, 4)) return GDR_ERR_MISALIGNED;
    a.dy = dy; a.dh_T = dh_T;
    a.du = du; a.ddelta = ddelta; a.dz = dz; a.dh0 = dh0;
    const size_t eg = dtype_size(grad_dtype);
    if (a.act_vec == kWhole && !aligned_to(dy, 4 * eg)) a.act_vec = kPairs;
    if (a.act_vec == kPairs && !aligned_to(dy, 2 * eg)) a.act_vec = kSingle;
    a.out_vec = a.K % 4 == 0 && aligned_to(du, 16) && aligned_to(ddelta, 16) && aligned_to(dz, 16);
    a.state_vec = states_in_quads(N, {A, h0, dh_T, dh0});
    return launched(launch_scan_bwd(a, workspace, dA, dB, dC, dD, ddelta_bias, B, dtype, grad_dtype,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

gdr_status gdr_scan_step(const void* u, const void* delta, const float* A, const void* Bm, const void* Cm,
                         const float* D, const void* z, const float* delta_bias, float* h, void* y,
                         const long long* strides, int B, int D_, int N, int G, int delta_softplus, int dtype,
                         void* stream) {
    long long s10[10];
    if (strides)
        for (int i = 0; i < 5; ++i) { s10[2 * i] = strides[i]; s10[2 * i + 1] = 0; }
    ScanArgs a;
    gdr_status ok = scan_fill(a, u, delta, A, Bm, Cm, D, z, delta_bias, h, nullptr, strides ? s10 : nullptr, false, B,
                              1, D_, N, G, delta_softplus, dtype);
    if (ok != GDR_OK) return ok;
    if (!h || !y) return GDR_ERR_INVALID_ARG;
    if (!aligned_to(y, dtype_size(dtype))) return GDR_ERR_MISALIGNED;
    a.y = y;
    a.state_vec = states_in_quads(N, {A, h});
    return launched(launch_scan_step(a, h, B, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
