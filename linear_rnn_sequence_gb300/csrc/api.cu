// api.cu -- the extern "C" entry points of liblinattn.so (declared in
// include/linattn.h): argument checks on the host, then dispatch to the
// kernels.  Nothing here computes attention; every step runs in the kernels.
#include <cmath>
#include <cstring>

#include "la_internal.h"

namespace la {

DebugFault &debug_fault() {
    static DebugFault f;
    return f;
}

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dim_ok(int x) { return x == 32 || x == 64 || x == 128; }

// [p, p+n) and [q, q+m) overlap?
bool overlap(const void *p, size_t n, const void *q, size_t m) {
    if (!p || !q || n == 0 || m == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

size_t esize(la_dtype dt) { return dt == LA_DTYPE_BF16 ? 2 : 4; }

la_status check_common(const void *q, const void *k, const void *v, const float *y, int B, int H,
                       long N, int d, int dv, la_dtype dt, float eps) {
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return LA_ERR_UNSUPPORTED;
    if (B < 1 || H < 1 || N < 0) return LA_ERR_INVALID_ARG;
    if (!dim_ok(d) || !dim_ok(dv)) return LA_ERR_UNSUPPORTED;
    if (!(eps > 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    const long long elems = (long long)B * H * (N > 0 ? N : 1) * (d > dv ? d : dv);
    if (elems >= (1LL << 31)) return LA_ERR_INVALID_ARG;
    const size_t es = esize(dt), T = (size_t)B * H * (N > 0 ? N : 0);
    if (T == 0) return LA_OK;  // no tokens: q, k, v, y are never touched (may be null)
    if (!q || !k || !v || !y) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(y)) return LA_ERR_INVALID_ARG;
    const size_t ybytes = T * dv * 4;
    if (overlap(y, ybytes, q, T * d * es) || overlap(y, ybytes, k, T * d * es) ||
        overlap(y, ybytes, v, T * dv * es))
        return LA_ERR_INVALID_ARG;
    return LA_OK;
}

la_status check_state(const float *S, const float *z, bool required) {
    if ((S == nullptr) != (z == nullptr)) return LA_ERR_INVALID_ARG;
    if (required && !S) return LA_ERR_INVALID_ARG;
    if (S && (!aligned16(S) || !aligned16(z))) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

la_status check_ws(void *ws, size_t have, size_t need) {
    if (need == 0) return LA_OK;
    if (!ws || have < need) return LA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LA_ERR_WORKSPACE;
    return LA_OK;
}

la_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

size_t causal_ws(int B, int H, int N, int d, int dv, la_dtype dt) {
    FwdArgs a{};
    a.B = B; a.H = H; a.N = N; a.d = d; a.dv = dv; a.dt = dt;
    if (B < 1 || H < 1 || N < 0 || !dim_ok(d) || !dim_ok(dv)) return 0;
    if (causal_tc_supported(a)) return causal_tc_workspace(B * H, N, d, dv);
    return 0;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

const char *la_status_string(la_status s) {
    switch (s) {
    case LA_OK: return "LA_OK";
    case LA_ERR_INVALID_ARG: return "LA_ERR_INVALID_ARG";
    case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED";
    case LA_ERR_CUDA: return "LA_ERR_CUDA";
    case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT";
    case LA_ERR_WORKSPACE: return "LA_ERR_WORKSPACE";
    }
    return "LA_ERR_UNKNOWN";
}

const char *la_version(void) { return "linattn 0.1 sm_103a"; }

size_t la_causal_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt) {
    return causal_ws(B, H, N, d, dv, dt);
}

size_t la_noncausal_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt) {
    if (B < 1 || H < 1 || N < 1 || !dim_ok(d) || !dim_ok(dv)) return 0;
    FwdArgs a{};
    a.B = B; a.H = H; a.N = N; a.d = d; a.dv = dv; a.dt = dt;
    if (noncausal_tc_supported(a)) return noncausal_tc_workspace(B * H, N, d, dv);
    return noncausal_simt_workspace(B * H, N, d, dv);
}

la_status la_forward_causal(const void *q, const void *k, const void *v, float *y, int B, int H,
                            int N, int d, int dv, la_dtype dt, float eps, const float *S_in,
                            const float *z_in, float *S_out, float *z_out, void *workspace,
                            size_t workspace_bytes, void *stream) {
    la_status st = check_common(q, k, v, y, B, H, N, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if ((st = check_state(S_in, z_in, false)) != LA_OK) return st;
    if ((st = check_state(S_out, z_out, false)) != LA_OK) return st;
    const size_t T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4, zb = (size_t)B * H * d * 4;
    if (overlap(y, T * dv * 4, S_in, sb) || overlap(y, T * dv * 4, z_in, zb) ||
        overlap(y, T * dv * 4, S_out, sb) || overlap(y, T * dv * 4, z_out, zb))
        return LA_ERR_INVALID_ARG;
    const size_t need = causal_ws(B, H, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (need > 0) {  // a fresh run-time status for every call that uses the workspace
        cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s);
        if (e != cudaSuccess) return LA_ERR_CUDA;
    }
    if (N == 0) {  // no tokens: the final state is the initial state
        if (S_out) {
            cudaError_t e = cudaSuccess;
            if (!S_in) e = cudaMemsetAsync(S_out, 0, sb, s);
            else if (S_in != S_out)
                e = cudaMemcpyAsync(S_out, S_in, sb, cudaMemcpyDeviceToDevice, s);
            if (e == cudaSuccess) {
                if (!z_in) e = cudaMemsetAsync(z_out, 0, zb, s);
                else if (z_in != z_out)
                    e = cudaMemcpyAsync(z_out, z_in, zb, cudaMemcpyDeviceToDevice, s);
            }
            return from_cuda(e);
        }
        return LA_OK;
    }
    FwdArgs a{q, k, v, y, B, H, N, d, dv, dt, eps, S_in, z_in, S_out, z_out,
              workspace, workspace_bytes, s};
    if (causal_tc_supported(a)) return from_cuda(launch_causal_tc(a));
    return from_cuda(launch_causal_simt(a));
}

la_status la_forward_noncausal(const void *q, const void *k, const void *v, float *y, int B,
                               int H, int N, int d, int dv, la_dtype dt, float eps, float *S_out,
                               float *z_out, void *workspace, size_t workspace_bytes,
                               void *stream) {
    la_status st = check_common(q, k, v, y, B, H, N, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if (N < 1) return LA_ERR_INVALID_ARG;
    if ((st = check_state(S_out, z_out, false)) != LA_OK) return st;
    const size_t T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4, zb = (size_t)B * H * d * 4;
    if (overlap(y, T * dv * 4, S_out, sb) || overlap(y, T * dv * 4, z_out, zb))
        return LA_ERR_INVALID_ARG;
    const size_t need = la_noncausal_workspace_bytes(B, H, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    FwdArgs a{q, k, v, y, B, H, N, d, dv, dt, eps, nullptr, nullptr, S_out, z_out,
              workspace, workspace_bytes, s};
    const bool tc = noncausal_tc_supported(a);
    // a fresh run-time status (and, on the tensor-core path, fresh per-head
    // counters) for every call
    if (cudaMemsetAsync(workspace, 0, tc ? noncausal_tc_clear_bytes(B * H) : sizeof(WsHeader), s) !=
        cudaSuccess)
        return LA_ERR_CUDA;
    if (tc) return from_cuda(launch_noncausal_tc(a));
    return from_cuda(launch_noncausal_simt(a));
}

la_status la_decode_step(const void *q, const void *k, const void *v, float *y, float *S,
                         float *z, int B, int H, int d, int dv, la_dtype dt, float eps,
                         void *stream) {
    la_status st = check_common(q, k, v, y, B, H, 1, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if ((st = check_state(S, z, true)) != LA_OK) return st;
    const size_t yb = (size_t)B * H * dv * 4, sb = (size_t)B * H * d * dv * 4,
                 zb = (size_t)B * H * d * 4;
    if (overlap(y, yb, S, sb) || overlap(y, yb, z, zb) || overlap(S, sb, z, zb))
        return LA_ERR_INVALID_ARG;
    DecodeArgs a{q, k, v, y, S, z, B, H, d, dv, dt, eps, static_cast<cudaStream_t>(stream)};
    return from_cuda(launch_decode_simt(a));
}

la_status la_forward_causal_decay(const void *q, const void *k, const void *v, float *y, int B,
                                  int H, int N, int d, int dv, la_dtype dt, float eps,
                                  const float *gamma, const float *S_in, const float *z_in,
                                  float *S_out, float *z_out, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    la_status st = check_common(q, k, v, y, B, H, N, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if (!gamma || (reinterpret_cast<uintptr_t>(gamma) & 3u) != 0) return LA_ERR_INVALID_ARG;
    if ((st = check_state(S_in, z_in, false)) != LA_OK) return st;
    if ((st = check_state(S_out, z_out, false)) != LA_OK) return st;
    const size_t T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4, zb = (size_t)B * H * d * 4;
    if (overlap(y, T * dv * 4, S_in, sb) || overlap(y, T * dv * 4, z_in, zb) ||
        overlap(y, T * dv * 4, S_out, sb) || overlap(y, T * dv * 4, z_out, zb) ||
        overlap(y, T * dv * 4, gamma, (size_t)H * 4))
        return LA_ERR_INVALID_ARG;
    const size_t need = causal_ws(B, H, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (need > 0) {  // a fresh run-time status for every call that uses the workspace
        if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    }
    if (N == 0) {  // no tokens: the final state is the initial state
        if (S_out) {
            cudaError_t e = cudaSuccess;
            if (!S_in) e = cudaMemsetAsync(S_out, 0, sb, s);
            else if (S_in != S_out)
                e = cudaMemcpyAsync(S_out, S_in, sb, cudaMemcpyDeviceToDevice, s);
            if (e == cudaSuccess) {
                if (!z_in) e = cudaMemsetAsync(z_out, 0, zb, s);
                else if (z_in != z_out)
                    e = cudaMemcpyAsync(z_out, z_in, zb, cudaMemcpyDeviceToDevice, s);
            }
            return from_cuda(e);
        }
        return LA_OK;
    }
    FwdArgs a{q, k, v, y, B, H, N, d, dv, dt, eps, S_in, z_in, S_out, z_out,
              workspace, workspace_bytes, s};
    a.gamma = gamma;
    // heads with decay_on_tensor_cores(gamma) on the tensor cores, then the
    // rest on the CUDA cores (the second kernel's CTAs for the first kind
    // return at once); no host read of gamma is needed to split them
    if (causal_tc_supported(a)) {
        const cudaError_t e = launch_causal_tc(a);
        if (e != cudaSuccess) return from_cuda(e);
        a.skip_tc_heads = true;
    }
    return from_cuda(launch_causal_simt(a));
}

la_status la_decode_step_decay(const void *q, const void *k, const void *v, float *y, float *S,
                               float *z, int B, int H, int d, int dv, la_dtype dt, float eps,
                               const float *gamma, void *stream) {
    la_status st = check_common(q, k, v, y, B, H, 1, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if (!gamma || (reinterpret_cast<uintptr_t>(gamma) & 3u) != 0) return LA_ERR_INVALID_ARG;
    if ((st = check_state(S, z, true)) != LA_OK) return st;
    const size_t yb = (size_t)B * H * dv * 4, sb = (size_t)B * H * d * dv * 4,
                 zb = (size_t)B * H * d * 4;
    if (overlap(y, yb, S, sb) || overlap(y, yb, z, zb) || overlap(S, sb, z, zb) ||
        overlap(gamma, (size_t)H * 4, S, sb) || overlap(gamma, (size_t)H * 4, z, zb) ||
        overlap(gamma, (size_t)H * 4, y, yb))
        return LA_ERR_INVALID_ARG;
    DecodeArgs a{q, k, v, y, S, z, B, H, d, dv, dt, eps, static_cast<cudaStream_t>(stream)};
    a.gamma = gamma;
    return from_cuda(launch_decode_simt(a));
}

size_t la_causal_gated_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt,
                                       la_phi phi, int gate_dim) {
    if (B < 1 || H < 1 || N < 0 || !dim_ok(d) || !dim_ok(dv)) return 0;
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return 0;
    if (gate_dim != 1 && gate_dim != d) return 0;
    FwdArgs a{};
    a.B = B; a.H = H; a.N = N; a.d = d; a.dv = dv; a.dt = dt;
    a.phi = (int)phi;
    a.gate = reinterpret_cast<const float *>(&a);   // a gate is given (its address is not used)
    a.gate_dim = gate_dim;
    if (N > 0 && gated_tc_supported(a)) return gated_tc_workspace(B * H, N, d, dv);
    return sizeof(WsHeader);
}

la_status la_forward_causal_gated(const void *q, const void *k, const void *v, float *y, int B,
                                  int H, int N, int d, int dv, la_dtype dt, float eps, la_phi phi,
                                  const float *gate, int gate_dim, const float *S_in,
                                  const float *z_in, float *S_out, float *z_out, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    la_status st = check_common(q, k, v, y, B, H, N, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if (phi != LA_PHI_ELU1 && phi != LA_PHI_IDENTITY) return LA_ERR_UNSUPPORTED;
    if (gate && gate_dim != 1 && gate_dim != d) return LA_ERR_INVALID_ARG;
    if (gate && (reinterpret_cast<uintptr_t>(gate) & 3u) != 0) return LA_ERR_INVALID_ARG;
    if ((st = check_state(S_in, z_in, false)) != LA_OK) return st;
    if ((st = check_state(S_out, z_out, false)) != LA_OK) return st;
    const size_t T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4, zb = (size_t)B * H * d * 4;
    const size_t gb = gate ? T * gate_dim * 4 : 0;
    if (overlap(y, T * dv * 4, S_in, sb) || overlap(y, T * dv * 4, z_in, zb) ||
        overlap(y, T * dv * 4, S_out, sb) || overlap(y, T * dv * 4, z_out, zb) ||
        overlap(y, T * dv * 4, gate, gb) || overlap(S_out, sb, gate, gb) ||
        overlap(z_out, zb, gate, gb))
        return LA_ERR_INVALID_ARG;
    const size_t need = gate ? la_causal_gated_workspace_bytes(B, H, N, d, dv, dt, phi, gate_dim)
                             : sizeof(WsHeader);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    if (overlap(workspace, need, y, T * dv * 4) || overlap(workspace, need, gate, gb) ||
        overlap(workspace, need, S_out, sb) || overlap(workspace, need, z_out, zb))
        return LA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // a fresh run-time status for every call (the tensor-core path also clears its flags)
    if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    if (N == 0) {  // no tokens: the final state is the initial state
        if (S_out) {
            cudaError_t e = cudaSuccess;
            if (!S_in) e = cudaMemsetAsync(S_out, 0, sb, s);
            else if (S_in != S_out)
                e = cudaMemcpyAsync(S_out, S_in, sb, cudaMemcpyDeviceToDevice, s);
            if (e == cudaSuccess) {
                if (!z_in) e = cudaMemsetAsync(z_out, 0, zb, s);
                else if (z_in != z_out)
                    e = cudaMemcpyAsync(z_out, z_in, zb, cudaMemcpyDeviceToDevice, s);
            }
            return from_cuda(e);
        }
        return LA_OK;
    }
    FwdArgs a{q, k, v, y, B, H, N, d, dv, dt, eps, S_in, z_in, S_out, z_out, workspace,
              workspace_bytes, s};
    a.phi = (int)phi;
    a.gate = gate;
    a.gate_dim = gate ? gate_dim : 1;
    return from_cuda(launch_causal_gated(a));
}

la_status la_decode_step_gated(const void *q, const void *k, const void *v, float *y, float *S,
                               float *z, int B, int H, int d, int dv, la_dtype dt, float eps,
                               la_phi phi, const float *gate, int gate_dim, void *stream) {
    la_status st = check_common(q, k, v, y, B, H, 1, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if (phi != LA_PHI_ELU1 && phi != LA_PHI_IDENTITY) return LA_ERR_UNSUPPORTED;
    if (gate && gate_dim != 1 && gate_dim != d) return LA_ERR_INVALID_ARG;
    if (gate && (reinterpret_cast<uintptr_t>(gate) & 3u) != 0) return LA_ERR_INVALID_ARG;
    if ((st = check_state(S, z, true)) != LA_OK) return st;
    const size_t yb = (size_t)B * H * dv * 4, sb = (size_t)B * H * d * dv * 4,
                 zb = (size_t)B * H * d * 4, gb = gate ? (size_t)B * H * gate_dim * 4 : 0;
    if (overlap(y, yb, S, sb) || overlap(y, yb, z, zb) || overlap(S, sb, z, zb) ||
        overlap(gate, gb, S, sb) || overlap(gate, gb, z, zb) || overlap(gate, gb, y, yb))
        return LA_ERR_INVALID_ARG;
    DecodeArgs a{q, k, v, y, S, z, B, H, d, dv, dt, eps, static_cast<cudaStream_t>(stream)};
    a.phi = (int)phi;
    a.gate = gate;
    a.gate_dim = gate ? gate_dim : 1;
    return from_cuda(launch_decode_simt(a));
}

size_t la_noncausal_phi_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt,
                                        la_phi phi) {
    if (phi == LA_PHI_ELU1) return la_noncausal_workspace_bytes(B, H, N, d, dv, dt);
    if (phi != LA_PHI_IDENTITY || B < 1 || H < 1 || N < 1 || !dim_ok(d) || !dim_ok(dv)) return 0;
    return noncausal_simt_workspace(B * H, N, d, dv);
}

la_status la_forward_noncausal_phi(const void *q, const void *k, const void *v, float *y, int B,
                                   int H, int N, int d, int dv, la_dtype dt, float eps,
                                   la_phi phi, float *S_out, float *z_out, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    if (phi == LA_PHI_ELU1)
        return la_forward_noncausal(q, k, v, y, B, H, N, d, dv, dt, eps, S_out, z_out, workspace,
                                    workspace_bytes, stream);
    if (phi != LA_PHI_IDENTITY) return LA_ERR_UNSUPPORTED;
    la_status st = check_common(q, k, v, y, B, H, N, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if (N < 1) return LA_ERR_INVALID_ARG;
    if ((st = check_state(S_out, z_out, false)) != LA_OK) return st;
    const size_t T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4, zb = (size_t)B * H * d * 4;
    if (overlap(y, T * dv * 4, S_out, sb) || overlap(y, T * dv * 4, z_out, zb))
        return LA_ERR_INVALID_ARG;
    const size_t need = la_noncausal_phi_workspace_bytes(B, H, N, d, dv, dt, phi);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    FwdArgs a{q, k, v, y, B, H, N, d, dv, dt, eps, nullptr, nullptr, S_out, z_out,
              workspace, workspace_bytes, s};
    a.phi = (int)phi;
    return from_cuda(launch_noncausal_simt(a));
}

la_status la_random_features(const void *x, float *phi_out, long long rows, int d, int m,
                             la_dtype dt, const float *W, void *stream) {
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return LA_ERR_UNSUPPORTED;
    if (rows < 0 || d < 1 || d > 128 || m < 1 || m > 256) return LA_ERR_INVALID_ARG;
    if (rows == 0) return LA_OK;
    if (!x || !phi_out || !W) return LA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(x) & (esize(dt) - 1)) != 0 ||
        (reinterpret_cast<uintptr_t>(phi_out) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(W) & 3u) != 0)
        return LA_ERR_INVALID_ARG;
    const size_t ob = (size_t)rows * m * 4;
    if (overlap(phi_out, ob, x, (size_t)rows * d * esize(dt)) ||
        overlap(phi_out, ob, W, (size_t)m * d * 4))
        return LA_ERR_INVALID_ARG;
    return from_cuda(launch_random_features(x, phi_out, rows, d, m, dt, W,
                                            static_cast<cudaStream_t>(stream)));
}

size_t la_causal_backward_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt) {
    if (B < 1 || H < 1 || N < 1 || !dim_ok(d) || !dim_ok(dv)) return 0;
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return 0;
    if ((long long)B * H * N * (d > dv ? d : dv) >= (1LL << 31)) return 0;
    return causal_backward_workspace(B * H, N, d, dv);
}

}  // extern "C"

namespace la {
namespace {

// la_backward_causal and la_backward_causal_decay (gamma null: no decay).
la_status backward_impl(const void *q, const void *k, const void *v, const float *dy,
                        float *grad_q, float *grad_k, float *grad_v, int B, int H, int N, int d,
                        int dv, la_dtype dt, float eps, const float *gamma, const float *S_in,
                        const float *z_in, float *grad_S_in, float *grad_z_in, void *workspace,
                        size_t workspace_bytes, void *stream) {
    la_status st = check_common(q, k, v, grad_v, B, H, N, d, dv, dt, eps);
    if (st != LA_OK) return st;
    if ((st = check_state(S_in, z_in, false)) != LA_OK) return st;
    if ((st = check_state(grad_S_in, grad_z_in, false)) != LA_OK) return st;
    const size_t BH = (size_t)B * H, T = BH * N, es = esize(dt);
    const size_t sb = BH * d * dv * 4, zb = BH * d * 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T > 0) {
        if (!dy || !grad_q || !grad_k) return LA_ERR_INVALID_ARG;
        if (!aligned16(dy) || !aligned16(grad_q) || !aligned16(grad_k)) return LA_ERR_INVALID_ARG;
    }
    const size_t need = la_causal_backward_workspace_bytes(B, H, N, d, dv, dt);
    // no output may overlap an input, the workspace or another output
    const struct { const void *p; size_t n; } outs[] = {
        {grad_q, T * d * 4}, {grad_k, T * d * 4}, {grad_v, T * dv * 4},
        {grad_S_in, grad_S_in ? sb : 0}, {grad_z_in, grad_z_in ? zb : 0}};
    const struct { const void *p; size_t n; } ins[] = {
        {q, T * d * es}, {k, T * d * es}, {v, T * dv * es}, {dy, T * dv * 4},
        {S_in, S_in ? sb : 0}, {z_in, z_in ? zb : 0}, {workspace, need}};
    for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
        for (const auto &in : ins)
            if (overlap(outs[i].p, outs[i].n, in.p, in.n)) return LA_ERR_INVALID_ARG;
        for (size_t j = i + 1; j < sizeof(outs) / sizeof(outs[0]); ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return LA_ERR_INVALID_ARG;
    }
    if (T == 0) {   // no tokens: the initial state gets no gradient
        if (grad_S_in) {
            cudaError_t e = cudaMemsetAsync(grad_S_in, 0, sb, s);
            if (e == cudaSuccess) e = cudaMemsetAsync(grad_z_in, 0, zb, s);
            return from_cuda(e);
        }
        return LA_OK;
    }
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    BwdArgs a{q, k, v, dy, grad_q, grad_k, grad_v, B, H, N, d, dv, dt, eps, S_in, z_in,
              grad_S_in, grad_z_in, workspace, workspace_bytes, s};
    a.gamma = gamma;
    return from_cuda(launch_causal_backward(a));
}

}  // namespace
}  // namespace la

extern "C" {

la_status la_backward_causal(const void *q, const void *k, const void *v, const float *dy,
                             float *grad_q, float *grad_k, float *grad_v, int B, int H, int N,
                             int d, int dv, la_dtype dt, float eps, const float *S_in,
                             const float *z_in, float *grad_S_in, float *grad_z_in,
                             void *workspace, size_t workspace_bytes, void *stream) {
    return backward_impl(q, k, v, dy, grad_q, grad_k, grad_v, B, H, N, d, dv, dt, eps, nullptr,
                         S_in, z_in, grad_S_in, grad_z_in, workspace, workspace_bytes, stream);
}

la_status la_backward_causal_decay(const void *q, const void *k, const void *v,
                                   const float *dy, float *grad_q, float *grad_k,
                                   float *grad_v, int B, int H, int N, int d, int dv,
                                   la_dtype dt, float eps, const float *gamma,
                                   const float *S_in, const float *z_in, float *grad_S_in,
                                   float *grad_z_in, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    if (!gamma || (reinterpret_cast<uintptr_t>(gamma) & 3u) != 0) return LA_ERR_INVALID_ARG;
    const size_t T = (size_t)B * H * (N > 0 ? N : 0);
    if (overlap(gamma, (size_t)H * 4, grad_q, T * d * 4) ||
        overlap(gamma, (size_t)H * 4, grad_k, T * d * 4) ||
        overlap(gamma, (size_t)H * 4, grad_v, T * dv * 4))
        return LA_ERR_INVALID_ARG;
    return backward_impl(q, k, v, dy, grad_q, grad_k, grad_v, B, H, N, d, dv, dt, eps, gamma,
                         S_in, z_in, grad_S_in, grad_z_in, workspace, workspace_bytes, stream);
}


// ---- gated delta rule, layer norm ------------------------------------------
}  // extern "C"

namespace la {
namespace {

struct Buf {
    const void *p;
    size_t n;
};
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Does any output overlap an input or another output?
template <int NI, int NO> bool clash(const Buf (&in)[NI], const Buf (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    }
    return false;
}

la_status check_delta(int B, int H, int Hk, long long N, int d, int dv, la_dtype dt) {
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return LA_ERR_UNSUPPORTED;
    if (B < 1 || H < 1 || Hk < 1 || N < 0 || H % Hk != 0) return LA_ERR_INVALID_ARG;
    if (!dim_ok(d) || !dim_ok(dv)) return LA_ERR_UNSUPPORTED;
    const long long BH = (long long)B * H, most = 1LL << 31;   // B*H below 2^62
    if (BH >= most || BH * d * dv >= most) return LA_ERR_INVALID_ARG;
    if (N > 0 && BH * (d > dv ? d : dv) >= (most + N - 1) / N) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

DeltaArgs delta_args(const void *q, const void *k, const void *v, const float *beta,
                     const float *log_gate, int B, int H, int Hk, int N, int d, int dv, la_dtype dt,
                     la_layout layout, const float *S_in, void *ws, void *stream) {
    DeltaArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.log_gate = log_gate;
    a.B = B; a.H = H; a.Hk = Hk; a.N = N; a.d = d; a.dv = dv; a.dt = dt; a.layout = layout;
    a.S_in = S_in; a.ws = ws; a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

size_t delta_bwd_ws_bytes(int B, int H, int Hk, int N, int d, int dv, la_dtype dt) {
    if (check_delta(B, H, Hk, N, d, dv, dt) != LA_OK || N == 0) return 0;
    return delta_backward_workspace(delta_args(nullptr, nullptr, nullptr, nullptr, nullptr, B, H, Hk, N,
                                               d, dv, dt, LA_LAYOUT_BHND, nullptr, nullptr, nullptr));
}

// The tensor-core kernel takes a block of 64 tokens at a time and has a longer start; below half a
// block the token-by-token kernel is done sooner.
bool delta_on_tensor_cores(const DeltaArgs &a) { return a.N >= 32 && delta_tc_supported(a); }

// dst = src, or zero without one.
cudaError_t copy_state(float *dst, const float *src, size_t bytes, cudaStream_t s) {
    if (!dst || dst == src) return cudaSuccess;
    if (!src) return cudaMemsetAsync(dst, 0, bytes, s);
    return cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s);
}

la_status check_norm(const void *x, const void *y, long long rows, int D, la_dtype dt) {
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return LA_ERR_UNSUPPORTED;
    if (rows < 0 || D < 1 || rows > (1LL << 62) / ((long long)D * 4)) return LA_ERR_INVALID_ARG;
    if (D > 16384) return LA_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !y)) return LA_ERR_INVALID_ARG;
    const uintptr_t m = esize(dt) - 1;
    if ((reinterpret_cast<uintptr_t>(x) & m) || (reinterpret_cast<uintptr_t>(y) & m))
        return LA_ERR_INVALID_ARG;
    return LA_OK;
}

}  // namespace
}  // namespace la

extern "C" {

size_t la_delta_workspace_bytes(int B, int H, int Hk, int N, int d, int dv, la_dtype dt) {
    if (check_delta(B, H, Hk, N, d, dv, dt) != LA_OK || N == 0) return 0;
    const DeltaArgs a = delta_args(nullptr, nullptr, nullptr, nullptr, nullptr, B, H, Hk, N, d, dv, dt,
                                   LA_LAYOUT_BHND, nullptr, nullptr, nullptr);
    return delta_on_tensor_cores(a) ? delta_tc_workspace(a) : 0;
}

la_status la_forward_delta(const void *q, const void *k, const void *v, void *y, const float *beta,
                           const float *log_gate, int B, int H, int Hk, int N, int d, int dv,
                           la_dtype dt, la_layout layout, const float *S_in, float *S_out,
                           void *workspace, size_t workspace_bytes, void *stream) {
    la_status st = check_delta(B, H, Hk, N, d, dv, dt);
    if (st != LA_OK) return st;
    if (layout != LA_LAYOUT_BHND && layout != LA_LAYOUT_BNHD) return LA_ERR_UNSUPPORTED;
    const size_t es = esize(dt), TH = (size_t)B * H * N, TK = (size_t)B * Hk * N;
    const size_t sb = (size_t)B * H * d * dv * 4;
    if (!aligned16(S_in) || !aligned16(S_out)) return LA_ERR_INVALID_ARG;
    if (S_in != S_out && overlap(S_in, sb, S_out, sb)) return LA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return from_cuda(copy_state(S_out, S_in, sb, s));   // no tokens: q .. beta may be NULL
    if (!q || !k || !v || !y || !beta) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(y) || !aligned4(beta) ||
        !aligned4(log_gate))
        return LA_ERR_INVALID_ARG;
    const size_t need = la_delta_workspace_bytes(B, H, Hk, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    const Buf in[] = {{q, TK * d * es}, {k, TK * d * es}, {v, TH * dv * es}, {beta, TH * 4},
                      {log_gate, TH * 4}, {S_in != S_out ? S_in : nullptr, sb}};
    const Buf out[] = {{y, TH * dv * es}, {S_out, sb}, {need ? workspace : nullptr, need}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    DeltaArgs a = delta_args(q, k, v, beta, log_gate, B, H, Hk, N, d, dv, dt, layout, S_in, workspace,
                             stream);
    a.y = y;
    a.S_out = S_out;
    if (need == 0) return from_cuda(launch_delta_forward_simt(a));
    if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    return from_cuda(launch_delta_forward_tc(a));
}

size_t la_delta_backward_workspace_bytes(int B, int H, int Hk, int N, int d, int dv, la_dtype dt) {
    return delta_bwd_ws_bytes(B, H, Hk, N, d, dv, dt);
}

la_status la_backward_delta(const void *q, const void *k, const void *v, const void *dy,
                            const float *beta, const float *log_gate, void *grad_q, void *grad_k,
                            void *grad_v, float *grad_beta, float *grad_log_gate, int B, int H, int Hk,
                            int N, int d, int dv, la_dtype dt, la_layout layout, const float *S_in,
                            const float *grad_S_out, float *grad_S_in, void *workspace,
                            size_t workspace_bytes, void *stream) {
    la_status st = check_delta(B, H, Hk, N, d, dv, dt);
    if (st != LA_OK) return st;
    if (layout != LA_LAYOUT_BHND && layout != LA_LAYOUT_BNHD) return LA_ERR_UNSUPPORTED;
    const size_t es = esize(dt), TH = (size_t)B * H * N, TK = (size_t)B * Hk * N;
    const size_t sb = (size_t)B * H * d * dv * 4;
    if (!aligned16(S_in) || !aligned16(grad_S_out) || !aligned16(grad_S_in)) return LA_ERR_INVALID_ARG;
    if (overlap(grad_S_in, sb, S_in, sb) || overlap(grad_S_in, sb, grad_S_out, sb))
        return LA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return from_cuda(copy_state(grad_S_in, grad_S_out, sb, s));
    const void *need16[] = {q, k, v, dy, grad_q, grad_k, grad_v};
    for (const void *p : need16)
        if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
    if (!beta || !grad_beta || (log_gate == nullptr) != (grad_log_gate == nullptr)) return LA_ERR_INVALID_ARG;
    if (!aligned4(beta) || !aligned4(log_gate) || !aligned4(grad_beta) || !aligned4(grad_log_gate))
        return LA_ERR_INVALID_ARG;
    const size_t need = delta_bwd_ws_bytes(B, H, Hk, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    const Buf in[] = {{q, TK * d * es}, {k, TK * d * es}, {v, TH * dv * es}, {dy, TH * dv * es},
                      {beta, TH * 4}, {log_gate, TH * 4}, {S_in, sb}, {grad_S_out, sb}};
    const Buf out[] = {{grad_q, TK * d * es}, {grad_k, TK * d * es}, {grad_v, TH * dv * es},
                       {grad_beta, TH * 4}, {grad_log_gate, TH * 4}, {grad_S_in, sb},
                       {workspace, need}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    DeltaArgs a = delta_args(q, k, v, beta, log_gate, B, H, Hk, N, d, dv, dt, layout, S_in, workspace,
                             stream);
    a.dy = dy;
    a.dq = grad_q; a.dk = grad_k; a.dv_grad = grad_v;
    a.dbeta = grad_beta; a.dlog_gate = grad_log_gate;
    a.dS_out = grad_S_out; a.dS_in = grad_S_in;
    return from_cuda(launch_delta_backward(a));
}

la_status la_decode_step_delta(const void *q, const void *k, const void *v, void *y, const float *beta,
                               const float *log_gate, const float *S_in, float *S_out, int B, int H,
                               int Hk, int d, int dv, la_dtype dt, void *stream) {
    la_status st = check_delta(B, H, Hk, 1, d, dv, dt);
    if (st != LA_OK) return st;
    const void *need16[] = {q, k, v, y, S_in, S_out};
    for (const void *p : need16)
        if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
    if (!beta || !aligned4(beta) || !aligned4(log_gate)) return LA_ERR_INVALID_ARG;
    const size_t es = esize(dt), TH = (size_t)B * H, TK = (size_t)B * Hk, sb = TH * d * dv * 4;
    const Buf in[] = {{q, TK * d * es}, {k, TK * d * es}, {v, TH * dv * es}, {beta, TH * 4},
                      {log_gate, TH * 4}, {S_in != S_out ? S_in : nullptr, sb}};
    const Buf out[] = {{y, TH * dv * es}, {S_out, sb}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    DeltaArgs a = delta_args(q, k, v, beta, log_gate, B, H, Hk, 1, d, dv, dt, LA_LAYOUT_BHND, S_in,
                             nullptr, stream);
    a.y = y;
    a.S_out = S_out;
    return from_cuda(launch_delta_step(a));
}

la_status la_layer_norm(const void *x, void *y, const float *weight, const float *bias, float *mean,
                        float *rstd, long long rows, int D, la_dtype dt, float eps, void *stream) {
    la_status st = check_norm(x, y, rows, D, dt);
    if (st != LA_OK) return st;
    if (!(eps > 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    if ((mean == nullptr) != (rstd == nullptr)) return LA_ERR_INVALID_ARG;
    if (!aligned4(weight) || !aligned4(bias) || !aligned4(mean) || !aligned4(rstd))
        return LA_ERR_INVALID_ARG;
    if (rows == 0) return LA_OK;
    const size_t n = (size_t)rows * D * esize(dt);
    const Buf in[] = {{x != y ? x : nullptr, n}, {weight, (size_t)D * 4}, {bias, (size_t)D * 4}};
    const Buf out[] = {{y, n}, {mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4}};
    const Buf same[] = {{x, n}};
    const Buf stats[] = {{mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4}};
    if (clash(in, out) || clash(same, stats)) return LA_ERR_INVALID_ARG;
    LayerNormArgs a{};
    a.x = x; a.y = y; a.weight = weight; a.bias = bias; a.mean = mean; a.rstd = rstd;
    a.rows = rows; a.D = D; a.dt = dt; a.eps = eps; a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(launch_layer_norm(a));
}

size_t la_layer_norm_backward_workspace_bytes(long long rows, int D, la_dtype dt) {
    if (rows < 1 || check_norm(&dt, &dt, rows, D, dt) != LA_OK) return 0;
    return layer_norm_partials(rows, D, dt) * 4;
}

la_status la_layer_norm_backward(const void *dy, const void *x, const float *mean, const float *rstd,
                                 const float *weight, void *grad_x, float *grad_weight,
                                 float *grad_bias, long long rows, int D, la_dtype dt, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    la_status st = check_norm(x, grad_x, rows, D, dt);
    if (st == LA_OK) st = check_norm(dy, dy, rows, D, dt);
    if (st != LA_OK) return st;
    if (!aligned4(weight) || !aligned4(mean) || !aligned4(rstd) || !aligned4(grad_weight) ||
        !aligned4(grad_bias))
        return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D * esize(dt), nr = (size_t)rows * 4, nd = (size_t)D * 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {   // empty sums
        cudaError_t e = grad_weight ? cudaMemsetAsync(grad_weight, 0, nd, s) : cudaSuccess;
        if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, nd, s);
        return from_cuda(e);
    }
    if (!mean || !rstd) return LA_ERR_INVALID_ARG;
    const bool sums = grad_weight || grad_bias;
    const size_t need = sums ? la_layer_norm_backward_workspace_bytes(rows, D, dt) : 0;
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    const Buf in[] = {{x != grad_x ? x : nullptr, n}, {dy != grad_x ? dy : nullptr, n},
                      {mean, nr}, {rstd, nr}, {weight, nd}};
    const Buf out[] = {{grad_x, n}, {grad_weight, nd}, {grad_bias, nd}, {sums ? workspace : nullptr, need}};
    const Buf whole[] = {{x, n}, {dy, n}};
    const Buf rest[] = {{grad_weight, nd}, {grad_bias, nd}, {sums ? workspace : nullptr, need}};
    if (clash(in, out) || clash(whole, rest)) return LA_ERR_INVALID_ARG;
    LayerNormArgs a{};
    a.x = x; a.dy = dy; a.dx = grad_x; a.weight = weight;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dweight = grad_weight; a.dbias = grad_bias;
    a.partials = sums ? static_cast<float *>(workspace) : nullptr;
    a.rows = rows; a.D = D; a.dt = dt; a.stream = s;
    return from_cuda(launch_layer_norm_backward(a));
}

}  // extern "C"

namespace la {
namespace {

// Rows of d elements at p + b st[0] + h st[1] + t st[2].
struct Rows {
    HeadsView v;
    long long n[3];   // batch rows, heads, tokens
    int d, es;
    long long st(int i) const { return i == 0 ? v.b : i == 1 ? v.h : v.t; }
    long long extent() const {   // elements from the first to the end of the last
        long long e = d;
        for (int i = 0; i < 3; ++i) e += (n[i] - 1) * st(i);
        return e;
    }
};

HeadsView heads_view(const void *p, const long long *st, la_layout layout, int heads, int N, int d) {
    HeadsView v{const_cast<void *>(p), 0, 0, 0};
    if (st) {
        v.b = st[0]; v.h = st[1]; v.t = st[2];
    } else if (layout == LA_LAYOUT_BHND) {
        v.b = (long long)heads * N * d; v.h = (long long)N * d; v.t = d;
    } else {
        v.b = (long long)N * heads * d; v.h = d; v.t = (long long)heads * d;
    }
    return v;
}

bool strides_ok(const Rows &r) {
    long long room = 1LL << 60;
    for (int i = 0; i < 3; ++i) {
        if (r.st(i) < 0) return false;
        if (r.n[i] > 1 && r.st(i) > room / (r.n[i] - 1)) return false;
        if (r.n[i] > 1) room -= (r.n[i] - 1) * r.st(i);
    }
    return room > 0;
}

// Order of the dimensions by the strides s, the widest first.
void widest_first(const long long (&s)[3], int (&o)[3]) {
    o[0] = 0; o[1] = 1; o[2] = 2;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (s[o[j]] < s[o[j + 1]]) { const int x = o[j]; o[j] = o[j + 1]; o[j + 1] = x; }
}

// May two rows of it share elements?
bool rows_overlap_each_other(const Rows &r) {
    const long long s[3] = {r.n[0] > 1 ? r.st(0) : 0, r.n[1] > 1 ? r.st(1) : 0, r.n[2] > 1 ? r.st(2) : 0};
    int o[3];
    widest_first(s, o);
    long long inner = r.d;
    for (int i = 2; i >= 0; --i) {
        if (r.n[o[i]] == 1) continue;
        if (s[o[i]] < inner) return true;
        inner += (r.n[o[i]] - 1) * s[o[i]];
    }
    return false;
}

// Does some row of b lie less than a row from some row of a, b's first being `at` elements behind a's?  Along the dimensions
// o[i] .. of common strides s, the widest first, only those steps count that the narrower dimensions can make up for.
bool rows_meet(const Rows &a, const Rows &b, const long long (&s)[3], const int (&o)[3], int i, long long at) {
    if (i == 3) return at < a.d && -at < a.d;
    const int x = o[i];
    if (s[x] == 0) return rows_meet(a, b, s, o, i + 1, at);
    long long up = a.d - 1, down = a.d - 1;   // narrower steps of a's and of b's, and a row
    for (int j = i + 1; j < 3; ++j) {
        up += (a.n[o[j]] - 1) * s[o[j]];
        down += (b.n[o[j]] - 1) * s[o[j]];
    }
    auto floored = [&](long long v) { return v >= 0 ? v / s[x] : -((-v + s[x] - 1) / s[x]); };
    long long first = -floored(at + down), last = floored(up - at);   // -down <= at + steps s <= up
    if (first < 1 - a.n[x]) first = 1 - a.n[x];
    if (last > b.n[x] - 1) last = b.n[x] - 1;
    if (last - first > 8) return first <= last;   // strides that are not nested (inputs): not looked into
    for (long long steps = first; steps <= last; ++steps)
        if (rows_meet(a, b, s, o, i + 1, at + steps * s[x])) return true;
    return false;
}

// May a row of a and a row of b share bytes?  Rows of other strides count as sharing what lies between their ends.
bool rows_overlap(const Rows &a, const Rows &b) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.v.p), pb = reinterpret_cast<uintptr_t>(b.v.p);
    if (pa > pb) return rows_overlap(b, a);
    if ((uintptr_t)a.extent() * a.es <= pb - pa) return false;
    if ((pb - pa) % a.es) return true;
    long long s[3];
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] > 1 && b.n[i] > 1 && a.st(i) != b.st(i)) return true;
        s[i] = a.n[i] > 1 ? a.st(i) : b.n[i] > 1 ? b.st(i) : 0;
    }
    int o[3];
    widest_first(s, o);
    return rows_meet(a, b, s, o, 0, (long long)((pb - pa) / a.es));
}

bool same_rows(const Rows &a, const Rows &b) {
    if (a.v.p != b.v.p) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.st(i) != b.st(i))) return false;
    return true;
}

bool overlap_rows(const Rows &r, const void *p, size_t bytes) {
    return overlap(r.v.p, (size_t)r.extent() * r.es, p, bytes);
}

la_status check_norm_rotate(int B, int Hq, int Hk, int N, int d, la_dtype dt) {
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16) return LA_ERR_UNSUPPORTED;
    if (B < 1 || Hq < 1 || Hk < 1 || N < 0 || Hq >= 65536 - (long long)Hk) return LA_ERR_INVALID_ARG;
    if (d < 2 || d > 256 || d % 2) return LA_ERR_UNSUPPORTED;
    if ((long long)B * N >= (1LL << 31)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

// Everything that both directions check; bufs: count / 2 tensors of q's heads and of k's in turn, the
// last two outputs.
la_status norm_rotate_args(NormRotateArgs &a, const void *const *bufs, int count, const long long *strides,
                           la_layout layout, const long long *positions, long long positions_stride) {
    la_status st = check_norm_rotate(a.B, a.Hq, a.Hk, a.N, a.d, a.dt);
    if (st != LA_OK) return st;
    if (layout != LA_LAYOUT_BHND && layout != LA_LAYOUT_BNHD) return LA_ERR_UNSUPPORTED;
    if (a.norm != LA_NORM_NONE && a.norm != LA_NORM_RMS && a.norm != LA_NORM_L2) return LA_ERR_UNSUPPORTED;
    if (a.pairs != LA_PAIRS_HALVES && a.pairs != LA_PAIRS_ADJACENT) return LA_ERR_UNSUPPORTED;
    if (a.norm != LA_NORM_NONE && (!(a.eps > 0.f) || !std::isfinite(a.eps))) return LA_ERR_INVALID_ARG;
    if (a.r < 0 || a.r > a.d / 2 || (a.r > 0 && !a.freq)) return LA_ERR_INVALID_ARG;
    const uintptr_t at8 = reinterpret_cast<uintptr_t>(a.r ? a.freq : nullptr) | reinterpret_cast<uintptr_t>(positions);
    if (!aligned4(a.wq) || !aligned4(a.wk) || (at8 & 7u)) return LA_ERR_INVALID_ARG;
    if (positions && (positions_stride < 0 || (a.B > 1 && positions_stride > (1LL << 59) / (a.B - 1)))) return LA_ERR_INVALID_ARG;
    if (a.N == 0) return LA_OK;
    const int es = (int)esize(a.dt);
    HeadsView *views[] = {&a.q, &a.k, &a.gq, &a.gk, &a.yq, &a.yk};
    Rows rows[6];
    for (int i = 0; i < count; ++i) {
        const int heads = i % 2 ? a.Hk : a.Hq;
        if (!bufs[i] || reinterpret_cast<uintptr_t>(bufs[i]) % es) return LA_ERR_INVALID_ARG;
        rows[i] = {heads_view(bufs[i], strides ? strides + 3 * i : nullptr, layout, heads, a.N, a.d), {a.B, heads, a.N}, a.d, es};
        if (!strides_ok(rows[i])) return LA_ERR_INVALID_ARG;
        for (int j = 0; j < 3; ++j)   // a stride that is not stepped along says nothing
            if (rows[i].n[j] == 1) (j == 0 ? rows[i].v.b : j == 1 ? rows[i].v.h : rows[i].v.t) = 0;
        *views[i < count - 2 ? i : i - count + 6] = rows[i].v;
    }
    const long long tokens = (a.B - 1) * positions_stride + a.N;
    for (int o = count - 2; o < count; ++o) {
        if (rows_overlap_each_other(rows[o])) return LA_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i) {
            const bool in_place = i < count - 2 && i % 2 == o % 2 && same_rows(rows[o], rows[i]);
            if (!in_place && rows_overlap(rows[o], rows[i])) return LA_ERR_INVALID_ARG;
        }
        if (overlap_rows(rows[o], a.wq, a.d * 4) || overlap_rows(rows[o], a.wk, a.d * 4) ||
            overlap_rows(rows[o], a.freq, (size_t)a.r * 8) || overlap_rows(rows[o], positions, (size_t)tokens * 8))
            return LA_ERR_INVALID_ARG;
    }
    a.positions = positions;
    a.pos_batch = positions_stride;
    return LA_OK;
}

NormRotateArgs rotate_args(int B, int Hq, int Hk, int N, int d, la_dtype dt, la_norm norm, float eps,
                           const float *wq, const float *wk, const double *freq, int rotated, la_pairs pairs,
                           void *stream) {
    NormRotateArgs a{};
    a.B = B; a.Hq = Hq; a.Hk = Hk; a.N = N; a.d = d; a.dt = dt; a.norm = norm; a.pairs = pairs; a.eps = eps;
    a.wq = wq; a.wk = wk; a.freq = freq; a.r = rotated; a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

}  // namespace
}  // namespace la

extern "C" {

la_status la_norm_rotate(const void *q, const void *k, void *q_out, void *k_out, const long long *strides, int B,
                         int Hq, int Hk, int N, int d, la_dtype dt, la_layout layout, la_norm norm, float eps,
                         const float *q_weight, const float *k_weight, const double *freq, int rotated,
                         la_pairs pairs, const long long *positions, long long positions_stride, void *stream) {
    NormRotateArgs a = rotate_args(B, Hq, Hk, N, d, dt, norm, eps, q_weight, k_weight, freq, rotated, pairs, stream);
    const void *bufs[] = {q, k, q_out, k_out};
    const la_status st = norm_rotate_args(a, bufs, 4, strides, layout, positions, positions_stride);
    if (st != LA_OK || N == 0) return st;
    return from_cuda(launch_norm_rotate(a));
}

size_t la_norm_rotate_backward_workspace_bytes(int B, int Hq, int Hk, int N, int d, la_dtype dt) {
    if (check_norm_rotate(B, Hq, Hk, N, d, dt) != LA_OK || N == 0) return 0;
    return norm_rotate_partials(rotate_args(B, Hq, Hk, N, d, dt, LA_NORM_RMS, 1.f, nullptr, nullptr, nullptr, 0,
                                            LA_PAIRS_HALVES, nullptr)) * 4;
}

la_status la_norm_rotate_backward(const void *q, const void *k, const void *gq_out, const void *gk_out, void *grad_q,
                                  void *grad_k, const long long *strides, int B, int Hq, int Hk, int N, int d,
                                  la_dtype dt, la_layout layout, la_norm norm, float eps, const float *q_weight,
                                  const float *k_weight, const double *freq, int rotated, la_pairs pairs,
                                  const long long *positions, long long positions_stride, float *grad_q_weight,
                                  float *grad_k_weight, void *workspace, size_t workspace_bytes, void *stream) {
    NormRotateArgs a = rotate_args(B, Hq, Hk, N, d, dt, norm, eps, q_weight, k_weight, freq, rotated, pairs, stream);
    const void *bufs[] = {q, k, gq_out, gk_out, grad_q, grad_k};
    la_status st = norm_rotate_args(a, bufs, 6, strides, layout, positions, positions_stride);
    if (st != LA_OK) return st;
    if (!aligned4(grad_q_weight) || !aligned4(grad_k_weight)) return LA_ERR_INVALID_ARG;
    const size_t nd = (size_t)d * 4;
    if (N == 0) {   // empty sums
        cudaError_t e = grad_q_weight ? cudaMemsetAsync(grad_q_weight, 0, nd, a.stream) : cudaSuccess;
        if (e == cudaSuccess && grad_k_weight) e = cudaMemsetAsync(grad_k_weight, 0, nd, a.stream);
        return from_cuda(e);
    }
    const bool sums = grad_q_weight || grad_k_weight;
    const size_t need = sums ? la_norm_rotate_backward_workspace_bytes(B, Hq, Hk, N, d, dt) : 0;
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    const Buf out[] = {{grad_q_weight, nd}, {grad_k_weight, nd}, {sums ? workspace : nullptr, need}};
    const Buf in[] = {{q_weight, nd}, {k_weight, nd}, {freq, (size_t)rotated * 8},
                      {positions, (size_t)((B - 1) * positions_stride + N) * 8}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    const HeadsView views[] = {a.q, a.k, a.gq, a.gk, a.yq, a.yk};
    for (int i = 0; i < 6; ++i) {
        const Rows r{views[i], {B, i % 2 ? Hk : Hq, N}, d, (int)esize(dt)};
        for (const Buf &o : out)
            if (overlap_rows(r, o.p, o.n)) return LA_ERR_INVALID_ARG;
    }
    a.dwq = grad_q_weight;
    a.dwk = grad_k_weight;
    a.partials = sums ? static_cast<float *>(workspace) : nullptr;
    return from_cuda(launch_norm_rotate_grad(a));
}

}  // extern "C"

namespace la {
namespace {

RetainArgs retain_args(const void *q, const void *k, const void *v, void *y, const float *gamma, int B, int H, int N,
                       int d, int dv, la_dtype dt, la_layout layout, const float *S_in, float *S_out, bool rev,
                       bool trans, void *ws, void *stream) {
    RetainArgs a{};
    a.q = q; a.k = k; a.v = v; a.y = y; a.gamma = gamma;
    a.B = B; a.H = H; a.N = N; a.d = d; a.dv = dv; a.dt = dt; a.layout = layout;
    a.S_in = S_in; a.S_out = S_out; a.rev = rev; a.trans = trans; a.ws = ws;
    a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

bool retain_on_tensor_cores(const RetainArgs &a) { return retain_tc_supported(a); }

// Of the forward, with a final state or without, or of the gradients.
size_t retain_ws_bytes(int B, int H, int N, int d, int dv, la_dtype dt, bool grads) {
    if (check_delta(B, H, H, N, d, dv, dt) != LA_OK || N == 0) return 0;
    float some;
    const RetainArgs a = retain_args(nullptr, nullptr, nullptr, nullptr, nullptr, B, H, N, d, dv, dt, LA_LAYOUT_BHND,
                                     nullptr, &some, false, false, nullptr, nullptr);
    return sizeof(WsHeader) + (retain_on_tensor_cores(a) ? retain_tc_workspace(a) : retain_simt_workspace(a, grads));
}

}  // namespace
}  // namespace la

extern "C" {

size_t la_retention_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt) {
    return retain_ws_bytes(B, H, N, d, dv, dt, false);
}

la_status la_forward_retention(const void *q, const void *k, const void *v, void *y, const float *gamma, int B, int H,
                               int N, int d, int dv, la_dtype dt, la_layout layout, const float *S_in, float *S_out,
                               void *workspace, size_t workspace_bytes, void *stream) {
    la_status st = check_delta(B, H, H, N, d, dv, dt);
    if (st != LA_OK) return st;
    if (layout != LA_LAYOUT_BHND && layout != LA_LAYOUT_BNHD) return LA_ERR_UNSUPPORTED;
    const size_t es = esize(dt), T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4;
    if (!aligned16(S_in) || !aligned16(S_out)) return LA_ERR_INVALID_ARG;
    if (S_in != S_out && overlap(S_in, sb, S_out, sb)) return LA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return from_cuda(copy_state(S_out, S_in, sb, s));   // no tokens: q .. gamma may be NULL
    if (!gamma || !aligned4(gamma)) return LA_ERR_INVALID_ARG;
    const void *need16[] = {q, k, v, y};
    for (const void *p : need16)
        if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
    const size_t need = la_retention_workspace_bytes(B, H, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    const Buf in[] = {{q, T * d * es}, {k, T * d * es}, {v, T * dv * es}, {gamma, (size_t)H * 4},
                      {S_in != S_out ? S_in : nullptr, sb}};
    const Buf out[] = {{y, T * dv * es}, {S_out, sb}, {need ? workspace : nullptr, need}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    if (need && cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    const RetainArgs a = retain_args(q, k, v, y, gamma, B, H, N, d, dv, dt, layout, S_in, S_out, false, false, workspace, stream);
    return from_cuda(retain_on_tensor_cores(a) ? launch_retain_tc(a) : launch_retain_simt(a));
}

size_t la_retention_backward_workspace_bytes(int B, int H, int N, int d, int dv, la_dtype dt) {
    return retain_ws_bytes(B, H, N, d, dv, dt, true);
}

la_status la_backward_retention(const void *q, const void *k, const void *v, const void *dy, const float *gamma,
                                void *grad_q, void *grad_k, void *grad_v, int B, int H, int N, int d, int dv,
                                la_dtype dt, la_layout layout, const float *S_in, const float *grad_S_out,
                                float *grad_S_in, void *workspace, size_t workspace_bytes, void *stream) {
    la_status st = check_delta(B, H, H, N, d, dv, dt);
    if (st != LA_OK) return st;
    if (layout != LA_LAYOUT_BHND && layout != LA_LAYOUT_BNHD) return LA_ERR_UNSUPPORTED;
    const size_t es = esize(dt), T = (size_t)B * H * N, sb = (size_t)B * H * d * dv * 4;
    if (!aligned16(S_in) || !aligned16(grad_S_out) || !aligned16(grad_S_in)) return LA_ERR_INVALID_ARG;
    if (overlap(grad_S_in, sb, S_in, sb) || overlap(grad_S_in, sb, grad_S_out, sb)) return LA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return from_cuda(copy_state(grad_S_in, grad_S_out, sb, s));
    if (!gamma || !aligned4(gamma)) return LA_ERR_INVALID_ARG;
    const void *need16[] = {q, k, v, dy, grad_q, grad_k, grad_v};
    for (const void *p : need16)
        if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
    const size_t need = la_retention_backward_workspace_bytes(B, H, N, d, dv, dt);
    if ((st = check_ws(workspace, workspace_bytes, need)) != LA_OK) return st;
    const Buf in[] = {{q, T * d * es}, {k, T * d * es}, {v, T * dv * es}, {dy, T * dv * es}, {gamma, (size_t)H * 4},
                      {S_in, sb}, {grad_S_out, sb}};
    const Buf out[] = {{grad_q, T * d * es}, {grad_k, T * d * es}, {grad_v, T * dv * es}, {grad_S_in, sb},
                       {need ? workspace : nullptr, need}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    if (need && cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return LA_ERR_CUDA;
    const RetainArgs a = retain_args(q, k, v, nullptr, gamma, B, H, N, d, dv, dt, layout, S_in, nullptr, false, false, workspace, stream);
    if (!retain_on_tensor_cores(a))
        return from_cuda(launch_retain_grads_simt(a, {dy, grad_q, grad_k, grad_v, grad_S_out, grad_S_in}));
    cudaError_t e = launch_retain_tc(retain_args(dy, v, k, grad_q, gamma, B, H, N, dv, d, dt, layout, S_in, nullptr, false, true, workspace, stream));
    if (e == cudaSuccess)
        e = launch_retain_tc(retain_args(k, q, dy, grad_v, gamma, B, H, N, d, dv, dt, layout, grad_S_out, grad_S_in, true, false, workspace, stream));
    if (e == cudaSuccess) {   // from the transposed state that grad_v's came from
        RetainArgs gk = retain_args(v, dy, q, grad_k, gamma, B, H, N, dv, d, dt, layout, grad_S_out, nullptr, true, true, workspace, stream);
        gk.have_states = true;
        e = launch_retain_tc(gk);
    }
    return from_cuda(e);
}

la_status la_decode_step_retention(const void *q, const void *k, const void *v, void *y, const float *gamma,
                                   const float *S_in, float *S_out, int B, int H, int d, int dv, la_dtype dt,
                                   void *stream) {
    la_status st = check_delta(B, H, H, 1, d, dv, dt);
    if (st != LA_OK) return st;
    const void *need16[] = {q, k, v, y, S_in, S_out};
    for (const void *p : need16)
        if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
    if (!gamma || !aligned4(gamma)) return LA_ERR_INVALID_ARG;
    const size_t es = esize(dt), T = (size_t)B * H, sb = T * d * dv * 4;
    const Buf in[] = {{q, T * d * es}, {k, T * d * es}, {v, T * dv * es}, {gamma, (size_t)H * 4},
                      {S_in != S_out ? S_in : nullptr, sb}};
    const Buf out[] = {{y, T * dv * es}, {S_out, sb}};
    if (clash(in, out)) return LA_ERR_INVALID_ARG;
    return from_cuda(launch_retain_step(retain_args(q, k, v, y, gamma, B, H, 1, d, dv, dt, LA_LAYOUT_BHND, S_in, S_out,
                                                    false, false, nullptr, stream)));
}

la_status la_workspace_status(const void *workspace, size_t workspace_bytes, void *stream) {
    if (!workspace || workspace_bytes < sizeof(WsHeader)) return LA_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return LA_ERR_CUDA;
    WsHeader h;
    if (cudaMemcpy(&h, workspace, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess)
        return LA_ERR_CUDA;
    return h.error == 0 ? LA_OK : static_cast<la_status>(h.error);
}

void la_debug_set_fault(int drop_load_item, long long wait_limit_ns) {
    debug_fault().drop_load_item = drop_load_item;
    debug_fault().wait_limit_ns = wait_limit_ns;
}

void la_debug_set_stall(long long ns) { debug_fault().stall_ns = ns < 0 ? 0 : ns > 1000000 ? 1000000 : ns; }

}  // extern "C"
