// C ABI of the low-rank adapters: argument checks and the launches (lora.cu).
#include <cstring>

#include "attn_checks.h"
#include "lora.h"
#include "sptp.h"

using namespace sptp;

namespace {

int check_lora(int P, int M, int K, int N, int R, int adapters, int rowwise) {
    if (P < 1 || P > kMaxGroups || M < 0 || M >= (1 << 30) || adapters < 0 || adapters >= (1 << 24)) return SPTP_ERR_SHAPE;
    if (R < 8 || R > kLoraMaxRank || R % 8 != 0) return SPTP_ERR_SHAPE;
    if (K < 8 || N < 8 || K > (1 << 20) || N > (1 << 20)) return SPTP_ERR_SHAPE;
    // a shard's part of the split dimension, and the other dimension, in rows of 16 bytes
    if (rowwise ? K % (8 * P) != 0 || N % 8 != 0 : N % (8 * P) != 0 || K % 8 != 0) return SPTP_ERR_SHAPE;
    const long long wide = static_cast<long long>(P) * (K > N ? K : N);
    return M <= (1ll << 42) / wide ? SPTP_OK : SPTP_ERR_SHAPE;
}

size_t lora_bytes(int P, int M, int K, int R, int rowwise, bool bf16) {
    int split_k;
    const int shards = rowwise ? P : 1;
    const size_t splits = lora_splits(M, K / shards, R, shards, bf16, &split_k);
    return SPTP_WS_HEADER_BYTES + align_up(splits * shards * M * R * sizeof(float));
}

}  // namespace

extern "C" {

size_t sptp_lora_workspace_size(int P, int M, int K, int N, int R, int rowwise) {
    if (check_lora(P, M, K, N, R, 0, rowwise) != SPTP_OK) return 0;
    const size_t a = lora_bytes(P, M, K, R, rowwise, true), b = lora_bytes(P, M, K, R, rowwise, false);
    return a > b ? a : b;
}

int sptp_lora(const void* x, const void* A, const void* B, const int* ids, const float* gains, int P, int M, int K, int N,
              int R, int adapters, int rowwise, sptp_dtype dtype, const void* base, void* out, void* workspace,
              size_t ws_bytes, void* cuda_stream) {
    return sptp_lora_ex(x, A, B, ids, gains, P, M, K, N, R, adapters, rowwise, dtype, base, out, workspace, ws_bytes, cuda_stream,
                        nullptr, 0);
}

int sptp_lora_ex(const void* x, const void* A, const void* B, const int* ids, const float* gains, int P, int M, int K, int N,
                 int R, int adapters, int rowwise, sptp_dtype dtype, const void* base, void* out, void* workspace,
                 size_t ws_bytes, void* cuda_stream, void* status_workspace, int check_only) {
    if (!workspace || (M != 0 && (!x || !ids || !base || !out || (adapters != 0 && (!A || !B))))) return SPTP_ERR_NULL;
    if (!dtype_ok(dtype)) return SPTP_ERR_DTYPE;
    int rc = check_lora(P, M, K, N, R, adapters, rowwise);
    if (rc != SPTP_OK) return rc;
    const size_t es = esize(dtype), m = static_cast<size_t>(M), n = static_cast<size_t>(adapters);
    const size_t need = sptp_lora_workspace_size(P, M, K, N, R, rowwise);
    const size_t out_bytes = (rowwise ? static_cast<size_t>(P) : 1) * m * N * es;
    const Buf ins[] = {{base, out_bytes, 16}, {x, m * K * es, 16}, {A, n * R * K * es, 16}, {B, n * N * R * es, 16},
                       {ids, m * 4, 4}, {gains, n * 4, 4}};
    const Buf outs[] = {{out, out_bytes, 16}, {workspace, need, kAlign}, {status_workspace, sizeof(DeviceStatus), kAlign}};
    const int n_outs = status_workspace ? 3 : 2;
    if ((rc = check_aligned(ins, 6)) != SPTP_OK || (rc = check_aligned(outs, n_outs)) != SPTP_OK) return rc;
    if (ws_bytes < need) return SPTP_ERR_WORKSPACE;
    const int skip = out == base ? 1 : 0;
    if ((rc = check_alias(outs, n_outs, ins + skip, 6 - skip)) != SPTP_OK) return rc;
    if (M == 0 || check_only) return SPTP_OK;
    DevInfo di;
    if ((rc = device_info(&di)) != SPTP_OK) return rc;
    LoraParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x;
    p.A = A;
    p.B = B;
    p.ids = ids;
    p.gains = gains;
    p.base = base;
    p.out = out;
    p.t = reinterpret_cast<float*>(mptr(workspace, SPTP_WS_HEADER_BYTES));
    p.P = P;
    p.M = M;
    p.K = K;
    p.N = N;
    p.R = R;
    p.adapters = adapters;
    p.rowwise = rowwise != 0;
    p.f = rowwise ? K / P : K;
    p.n = rowwise ? N : N / P;
    p.splits = lora_splits(M, p.f, R, rowwise ? P : 1, dtype == SPTP_BF16, &p.split_k);
    p.status = ws_status(status_workspace ? status_workspace : workspace);
    p.beside = status_workspace != nullptr;
    return cuda_status(launch_lora(p, dtype == SPTP_BF16, di.sms, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
