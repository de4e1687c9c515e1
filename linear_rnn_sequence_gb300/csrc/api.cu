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
