// serve_dispatch.cu -- picks the kernel of the serving-step calls.
#include "chunk_plan.cuh"
#include "serve.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"

namespace spd {

namespace {
// 0 the specialised kernel where the shapes and layouts allow it, 1 the
// general-layout kernel; index 0 = stage 5 (prefill attention), 1 = stage 6
thread_local int g_serve_policy[2] = {0, 0};
}  // namespace

int set_serve_policy(int stage, int policy) {
    if (stage < 5 || stage > 6) return -1;
    const int old = g_serve_policy[stage - 5];
    g_serve_policy[stage - 5] = policy;
    return old;
}

cudaError_t dispatch_store(const StoreArgs &a, cudaStream_t stream) {
    if (g_serve_policy[1] == 0) {
        bool used = false;
        const cudaError_t e = launch_store_vec(a, stream, &used);
        if (e != cudaSuccess || used) return e;
    }
    return launch_store_generic(a, stream);
}

cudaError_t dispatch_chunk(const ChunkArgs &a, void *ws, size_t ws_bytes, cudaStream_t stream) {
    (void)ws_bytes;
    if (g_serve_policy[0] == 0) {
        bool used = false;
        const cudaError_t e = launch_chunk_tc(a, ws, stream, &used);
        if (e != cudaSuccess || used) return e;
    }
    const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int32_t), stream);  // the status word
    if (e != cudaSuccess) return e;
    return launch_chunk_generic(a, stream);
}

size_t chunk_workspace_bytes(int64_t total_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t NB,
                             int64_t n_rows) {
    return ChunkLayout(total_q, Hq, Hkv, D, B, NB, n_rows).total;
}

}  // namespace spd
