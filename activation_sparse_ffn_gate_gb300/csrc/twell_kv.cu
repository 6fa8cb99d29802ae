// twell_kv.cu -- the paged key-value cache: new tokens' keys and values written to their slots
// (copied as bf16, or rounded to e4m3 with one fp32 scale per token and head), and slots read back
// as bf16.
//
// Both are bounded by memory traffic. A row (one token's key and value of one head) is handled by
// head_dim / 8 neighbouring lanes, 16 bytes of bf16 a lane, key and value in flight together; the
// row's largest magnitude is a shuffle over those lanes, so a row is read once.
#include "twell_kv.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kKvThreads = 256;

// The row of this thread: `lpr` lanes a row (a power of two, head_dim / 8 of them active).
struct KvRow {
    int token, head, col;
    bool live;
};
template <int LPR>
__device__ __forceinline__ KvRow kv_row(int n, int heads, int hd)
{
    const unsigned id = blockIdx.x * (kKvThreads / LPR) + threadIdx.x / LPR;
    KvRow r;
    r.col = static_cast<int>(threadIdx.x % LPR) * 8;
    r.token = static_cast<int>(id / static_cast<unsigned>(heads));
    r.head = static_cast<int>(id % static_cast<unsigned>(heads));
    r.live = r.token < n && r.col < hd;
    return r;
}

// The slot of a token: -1 where it has none or the slot does not exist (which is recorded).
__device__ __forceinline__ int checked_slot(const int32_t* slots, int token, const KvView& c, int32_t* status)
{
    const int s = slots[token];
    if (s >= 0 && (s >> c.page_shift) < c.n_pages) return s;
    if (s != -1) report(status, TWELL_ERR_DEVICE_CHECK);
    return -1;
}

template <int LPR, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvView c, const __nv_bfloat16* __restrict__ k,
                                                               const __nv_bfloat16* __restrict__ v, int64_t ldk,
                                                               int64_t ldv, const int32_t* __restrict__ slots, int n,
                                                               int32_t* status)
{
    pdl_begin();
    const KvRow r = kv_row<LPR>(n, c.heads, c.hd);
    uint4 kv[2] = {};
    int slot = -1;
    if (r.live) {
        const int64_t in = static_cast<int64_t>(r.head) * c.hd + r.col;
        kv[0] = ldg_stream16(k + r.token * ldk + in);
        kv[1] = ldg_stream16(v + r.token * ldv + in);
        slot = checked_slot(slots, r.token, c, status);
    }
    const int64_t off = slot >= 0 ? c.row(slot, r.head) + r.col : 0;
    if constexpr (!Q8) {
        if (slot < 0) return;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.k) + off) = kv[0];
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.v) + off) = kv[1];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[8];
            unpack16(kv[i], x, static_cast<__nv_bfloat16*>(nullptr));
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (slot < 0) continue;
            const Scale8 q(top);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(i == 0 ? c.k : c.v) + off) = q.pack8(x);
            if (r.col == 0) (i == 0 ? c.k_scale : c.v_scale)[c.scale_row(slot, r.head)] = q.scale;
        }
    }
}

template <int LPR, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_gather_kernel(const KvView c, const int32_t* __restrict__ slots, int n,
                                                               __nv_bfloat16* __restrict__ k_out,
                                                               __nv_bfloat16* __restrict__ v_out, int32_t* status)
{
    pdl_begin();
    const KvRow r = kv_row<LPR>(n, c.heads, c.hd);
    if (!r.live) return;
    const int slot = checked_slot(slots, r.token, c, status);
    const int64_t out = (static_cast<int64_t>(r.token) * c.heads + r.head) * c.hd + r.col;
    uint4 kv[2] = {};
    if (slot >= 0) {
        const int64_t off = c.row(slot, r.head) + r.col;
        if constexpr (!Q8) {
            kv[0] = ldg_stream16(static_cast<const __nv_bfloat16*>(c.k) + off);
            kv[1] = ldg_stream16(static_cast<const __nv_bfloat16*>(c.v) + off);
        } else {
            const int64_t so = c.scale_row(slot, r.head);
            const uint2 kc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + off));
            const uint2 vc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + off));
            const float s[2] = {__ldg(c.k_scale + so), __ldg(c.v_scale + so)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint2 q = i == 0 ? kc : vc;
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = e < 2 ? q.x : q.y;
                    const float2 p = e4m3x2_f32(static_cast<uint16_t>(e & 1 ? w >> 16 : w & 0xffffu));
                    x[2 * e] = p.x * s[i];
                    x[2 * e + 1] = p.y * s[i];
                }
                kv[i] = pack16(x, static_cast<__nv_bfloat16*>(nullptr));
            }
        }
    }
    *reinterpret_cast<uint4*>(k_out + out) = kv[0];
    *reinterpret_cast<uint4*>(v_out + out) = kv[1];
}

template <int LPR>
twell_status run_append(const KvView& c, const void* k, const void* v, int64_t ldk, int64_t ldv, const int32_t* slots,
                        int n, int32_t* status, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    const long long rows = static_cast<long long>(n) * c.heads;
    const int per = kKvThreads / LPR;
    auto kern = c.q8 ? kv_append_kernel<LPR, true> : kv_append_kernel<LPR, false>;
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kKvThreads), 0, s, c,
                                  static_cast<const bf*>(k), static_cast<const bf*>(v), ldk, ldv, slots, n, status);
}

template <int LPR>
twell_status run_gather(const KvView& c, const int32_t* slots, int n, void* k_out, void* v_out, int32_t* status,
                        cudaStream_t s)
{
    using bf = __nv_bfloat16;
    const long long rows = static_cast<long long>(n) * c.heads;
    const int per = kKvThreads / LPR;
    auto kern = c.q8 ? kv_gather_kernel<LPR, true> : kv_gather_kernel<LPR, false>;
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kKvThreads), 0, s, c,
                                  slots, n, static_cast<bf*>(k_out), static_cast<bf*>(v_out), status);
}

constexpr long long kMaxRows = 1ll << 31;  // rows (tokens x heads) of one call

}  // namespace
}  // namespace twell

using namespace twell_host;

twell_status twell_host::check_kv(const twell_kv_cache* c, twell::KvView* out)
{
    if (c == nullptr) return TWELL_ERR_INVALID;
    if (c->n_pages < 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0) return TWELL_ERR_INVALID;
    if (c->dtype != TWELL_BF16 && c->dtype != TWELL_E4M3) return TWELL_ERR_UNSUPPORTED;
    if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size > 1024 || c->head_dim % 16 != 0 || c->head_dim > 256 ||
        static_cast<long long>(c->n_pages) * c->page_size > INT32_MAX)
        return TWELL_ERR_UNSUPPORTED;
    const bool q8 = c->dtype == TWELL_E4M3;
    const int per16 = q8 ? 16 : 8;
    const int64_t strides[3] = {c->page_stride, c->head_stride, c->token_stride};
    for (int64_t s : strides)
        if (s < 0 || s % per16 != 0) return TWELL_ERR_INVALID;
    if (c->token_stride < c->head_dim && c->page_size > 1) return TWELL_ERR_INVALID;
    if (q8 && (c->scale_page_stride < 0 || c->scale_head_stride < 0)) return TWELL_ERR_INVALID;
    if (c->n_pages > 0) {
        if (c->k == nullptr || c->v == nullptr || !aligned16(c->k) || !aligned16(c->v)) return TWELL_ERR_INVALID;
        if (q8 && (c->k_scale == nullptr || c->v_scale == nullptr)) return TWELL_ERR_INVALID;
    }
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    *out = twell::KvView{c->k,           c->v,           c->k_scale,      c->v_scale,           c->page_stride,
                         c->head_stride, c->token_stride, c->scale_page_stride, c->scale_head_stride, c->n_pages,
                         shift,          c->n_kv_heads,  c->head_dim,     q8 ? 1 : 0};
    return TWELL_OK;
}

extern "C" twell_status twell_kv_append(const twell_kv_cache* cache, const void* k, const void* v, int64_t ldk,
                                        int64_t ldv, const int32_t* slots, int32_t n, int32_t* dev_status,
                                        void* stream)
{
    twell::KvView c;
    twell_status st = check_kv(cache, &c);
    if (st != TWELL_OK) return st;
    if (n < 0 || dev_status == nullptr) return TWELL_ERR_INVALID;
    if (n == 0) return TWELL_OK;
    const int64_t row = static_cast<int64_t>(c.heads) * c.hd;
    if (k == nullptr || v == nullptr || slots == nullptr || !aligned16(k) || !aligned16(v) || ldk % 8 != 0 ||
        ldv % 8 != 0 || ldk < row || ldv < row)
        return TWELL_ERR_INVALID;
    if (static_cast<long long>(n) * c.heads >= twell::kMaxRows) return TWELL_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.hd <= 64) return twell::run_append<8>(c, k, v, ldk, ldv, slots, n, dev_status, s);
    if (c.hd <= 128) return twell::run_append<16>(c, k, v, ldk, ldv, slots, n, dev_status, s);
    return twell::run_append<32>(c, k, v, ldk, ldv, slots, n, dev_status, s);
}

extern "C" twell_status twell_kv_gather(const twell_kv_cache* cache, const int32_t* slots, int32_t n, void* k_out,
                                        void* v_out, int32_t* dev_status, void* stream)
{
    twell::KvView c;
    twell_status st = check_kv(cache, &c);
    if (st != TWELL_OK) return st;
    if (n < 0 || dev_status == nullptr) return TWELL_ERR_INVALID;
    if (n == 0) return TWELL_OK;
    if (slots == nullptr || k_out == nullptr || v_out == nullptr || !aligned16(k_out) || !aligned16(v_out))
        return TWELL_ERR_INVALID;
    if (static_cast<long long>(n) * c.heads >= twell::kMaxRows) return TWELL_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.hd <= 64) return twell::run_gather<8>(c, slots, n, k_out, v_out, dev_status, s);
    if (c.hd <= 128) return twell::run_gather<16>(c, slots, n, k_out, v_out, dev_status, s);
    return twell::run_gather<32>(c, slots, n, k_out, v_out, dev_status, s);
}
