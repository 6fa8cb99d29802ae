// twell_lora.cu -- low-rank adapters of many requests beside a shared projection: to each token's row y the product
// s B (A x) of its own adapter (or of none) is added, A [R, k] and B [n, R] of bf16.
//
// One block a token: A x in fp32 by warps, a row of A each, then B's rows against it.
#include "twell_common.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = 4096;
constexpr int kLoraMaxTokens = 1 << 20;
constexpr int kLoraMaxDim = 1 << 20;
constexpr int kLoraThreads = 256;

struct LoraArgs {
    const __nv_bfloat16 *a, *b, *x, *y;
    __nv_bfloat16* out;
    const float* scale;
    const int32_t *ranks, *ids;
    int32_t* status;
    int64_t ldx, ldy, ldo;
    int L, R, k, n, N;
};

__global__ void __launch_bounds__(kLoraThreads) lora_kernel(const LoraArgs g)
{
    __shared__ float t[kLoraMaxRank];
    pdl_begin();
    const int tok = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int id = g.ids[tok];
    if (id < -1 || id >= g.L) {
        report(g.status, TWELL_ERR_DEVICE_CHECK);
        id = -1;
    }
    const __nv_bfloat16* y = g.y + tok * g.ldy;
    __nv_bfloat16* out = g.out + tok * g.ldo;
    int rank = 0;
    if (id >= 0) {
        rank = g.ranks ? g.ranks[id] : g.R;
        if (rank < 0 || rank > g.R) {
            report(g.status, TWELL_ERR_DEVICE_CHECK);
            rank = 0;
        }
    }
    if (rank == 0 && g.y == g.out) return;
    for (int r = warp; r < rank; r += kLoraThreads / 32) {
        const __nv_bfloat16* row = g.a + (static_cast<int64_t>(id) * g.R + r) * g.k;
        float sum = 0.0f;
        for (int c = lane * 8; c < g.k; c += 256) {
            float u[8], v[8];
            load8(row + c, u);
            load8(g.x + tok * g.ldx + c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(u[e], v[e], sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) t[r] = sum * g.scale[id];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < g.n; c += kLoraThreads) {
        const __nv_bfloat16* row = g.b + (static_cast<int64_t>(id) * g.n + c) * g.R;
        float sum = 0.0f;
        for (int r = 0; r < rank; ++r) sum = fmaf(__bfloat162float(row[r]), t[r], sum);
        out[c] = rank ? __float2bfloat16_rn(__bfloat162float(y[c]) + sum) : y[c];
    }
}

}  // namespace
}  // namespace twell

using namespace twell_host;

size_t twell_host::lora_ws_bytes(int N)
{
    (void)N;
    return 0;
}

extern "C" twell_status twell_lora_add(const void* y, int64_t ldy, const void* x, int64_t ldx, const twell_adapters* ad,
                                       const int32_t* ids, int32_t N, void* out, int64_t ldo, void* ws, size_t ws_bytes,
                                       int32_t* dev_status, void* stream)
{
    if (ad == nullptr || N < 0 || ad->n_adapters <= 0 || ad->rank <= 0 || ad->k <= 0 || ad->n <= 0 || ad->rank % 8 != 0 ||
        ad->k % 8 != 0 || ad->n % 8 != 0)
        return TWELL_ERR_INVALID;
    if (ad->rank > twell::kLoraMaxRank || ad->n_adapters > twell::kLoraMaxAdapters || N > twell::kLoraMaxTokens ||
        ad->k > twell::kLoraMaxDim || ad->n > twell::kLoraMaxDim)
        return TWELL_ERR_UNSUPPORTED;
    if (N == 0) return TWELL_OK;
    const void* need[] = {y, x, ad->a, ad->b, ad->scale, ids, out, dev_status};
    for (const void* p : need)
        if (p == nullptr) return TWELL_ERR_INVALID;
    const void* rows[] = {y, x, ad->a, ad->b, out};
    for (const void* p : rows)
        if (!aligned16(p)) return TWELL_ERR_INVALID;
    const void* words[] = {ad->scale, ad->ranks, ids};
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) % sizeof(int32_t) != 0) return TWELL_ERR_INVALID;
    if (ldy % 8 != 0 || ldx % 8 != 0 || ldo % 8 != 0 || ldy < ad->n || ldx < ad->k || ldo < ad->n) return TWELL_ERR_INVALID;
    if (y == out && ldy != ldo) return TWELL_ERR_INVALID;
    const size_t need_ws = lora_ws_bytes(N);
    if (need_ws > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < need_ws)) return TWELL_ERR_WORKSPACE;
    using bf = __nv_bfloat16;
    const twell::LoraArgs g = {static_cast<const bf*>(ad->a), static_cast<const bf*>(ad->b), static_cast<const bf*>(x),
                               static_cast<const bf*>(y), static_cast<bf*>(out), ad->scale, ad->ranks, ids, dev_status,
                               ldx, ldy, ldo, ad->n_adapters, ad->rank, ad->k, ad->n, N};
    return launch_dep(twell::lora_kernel, dim3(N), dim3(twell::kLoraThreads), 0, static_cast<cudaStream_t>(stream), g);
}
