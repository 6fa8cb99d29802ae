// twell_kv.cu -- the paged key-value cache: new tokens' keys and values written to their slots
// (copied as bf16, or rounded to e4m3 with one fp32 scale per token and head), and slots read back
// as bf16.
//
// Both are bounded by memory traffic. A row (one token's key and value of one head) is handled by
// neighbouring lanes, key and value in flight together. Writing: head_dim / 8 lanes, 16 bytes of bf16 a lane; the
// row's largest magnitudes are a shuffle over those lanes (key and value as one bf16 pair), and the four
// quotients of a row (both scales and both factors) are formed by different lanes with one division. Reading:
// head_dim / 8 lanes, so that a warp's 16-byte stores are contiguous, and with many rows kGatherRows rows a thread,
// all requested before the first is used.
#include "twell_kv.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kKvThreads = 256;
constexpr int kGatherRows = 4;

// Row `i` of this thread: LPR lanes a row (a power of two), 8 elements a lane, the lanes past head_dim idle. The rows of a
// block are one head's of consecutive tokens: neighbours in a page of the cache.
struct KvRow {
    int token, head, col;
    bool live;
};
template <int LPR, int RPT>
__device__ __forceinline__ KvRow kv_row(int i, int n, int heads, int hd)
{
    constexpr unsigned kPer = kKvThreads / LPR;
    const unsigned unit = blockIdx.x * RPT + i, tile = unit / static_cast<unsigned>(heads);
    KvRow r;
    r.col = static_cast<int>(threadIdx.x % LPR) * 8;
    r.head = static_cast<int>(unit - tile * heads);
    r.token = static_cast<int>(tile * kPer + threadIdx.x / LPR);
    r.live = r.token < n && r.col < hd;
    return r;
}

// A token's slot, -1 where it has none or the slot does not exist (which is recorded).
__device__ __forceinline__ int checked_slot(int s, const KvView& c, int32_t* status)
{
    if (s >= 0 && (s >> c.page_shift) < c.n_pages) return s;
    if (s != -1) report(status, TWELL_ERR_DEVICE_CHECK);
    return -1;
}

// The largest magnitude of 8 bf16 values, as a bf16 pair of which either may be it (NaN ignored).
__device__ __forceinline__ __nv_bfloat162 top8(const uint4& v)
{
    const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(w);
    return __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
}

template <int LPR, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvView c, const __nv_bfloat16* __restrict__ k,
                                                               const __nv_bfloat16* __restrict__ v, int64_t ldk,
                                                               int64_t ldv, const int32_t* __restrict__ slots, int n,
                                                               int32_t* status)
{
    pdl_begin();
    const KvRow r = kv_row<LPR, 1>(0, n, c.heads, c.hd);
    uint4 kv[2] = {};
    int slot = -1;
    if (r.live) {
        const int64_t in = static_cast<int64_t>(r.head) * c.hd + r.col;
        kv[0] = ldg_stream16(k + r.token * ldk + in);
        kv[1] = ldg_stream16(v + r.token * ldv + in);
        slot = checked_slot(__ldg(slots + r.token), c, status);
    }
    const int64_t off = slot >= 0 ? c.row(slot, r.head) + r.col : 0;
    if constexpr (!Q8) {
        if (slot < 0) return;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.k) + off) = kv[0];
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.v) + off) = kv[1];
    } else {
        const __nv_bfloat162 tk = top8(kv[0]), tv = top8(kv[1]);
        __nv_bfloat162 top = __hmax2(__lows2bfloat162(tk, tv), __highs2bfloat162(tk, tv));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = __hmax2(top, __shfl_xor_sync(0xffffffffu, top, o));
        // quarters of the row's lanes: the key's scale, its factor, the value's scale, its factor
        const int lane = threadIdx.x % LPR, part = lane / (LPR / 4);
        const float a = fmaxf(part < 2 ? __low2float(top) : __high2float(top), kAmaxMin);
        const float num = (part & 1) ? kE4m3Max : a, den = (part & 1) ? a : kE4m3Max;
        const float quot = num / den;
        const int row0 = static_cast<int>(threadIdx.x & 31) - lane;
        const float mk = __shfl_sync(0xffffffffu, quot, row0 + LPR / 4);
        const float mv = __shfl_sync(0xffffffffu, quot, row0 + 3 * (LPR / 4));
        // the lanes that hold the scales may lie past head_dim: they take the slot from the row's first lane
        const int row_slot = __shfl_sync(0xffffffffu, slot, row0);
        if (row_slot >= 0 && (lane == 0 || lane == LPR / 2))
            (lane == 0 ? c.k_scale : c.v_scale)[c.scale_row(row_slot, r.head)] = quot;
        if (slot < 0) return;
        float x[8];
        unpack16(kv[0], x, static_cast<__nv_bfloat16*>(nullptr));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.k) + off) = Scale8{0.0f, mk}.pack8(x);
        unpack16(kv[1], x, static_cast<__nv_bfloat16*>(nullptr));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.v) + off) = Scale8{0.0f, mv}.pack8(x);
    }
}

template <int LPR, bool Q8, int RPT>
__global__ void __launch_bounds__(kKvThreads) kv_gather_kernel(const KvView c, const int32_t* __restrict__ slots, int n,
                                                               __nv_bfloat16* __restrict__ k_out,
                                                               __nv_bfloat16* __restrict__ v_out, int32_t* status)
{
    pdl_begin();
    int slot[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const KvRow r = kv_row<LPR, RPT>(i, n, c.heads, c.hd);
        slot[i] = r.live ? __ldg(slots + r.token) : -1;
    }
    uint4 kv[RPT][2];  // an e4m3 row: its 8 codes in x and y, its scale in z
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const KvRow r = kv_row<LPR, RPT>(i, n, c.heads, c.hd);
        const int s = checked_slot(slot[i], c, status);
        kv[i][0] = kv[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (s < 0) continue;
        const int64_t off = c.row(s, r.head) + r.col;
        if constexpr (!Q8) {
            kv[i][0] = ldg_stream16(static_cast<const __nv_bfloat16*>(c.k) + off);
            kv[i][1] = ldg_stream16(static_cast<const __nv_bfloat16*>(c.v) + off);
        } else {
            const int64_t so = c.scale_row(s, r.head);
            const uint2 kc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + off));
            const uint2 vc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + off));
            kv[i][0] = make_uint4(kc.x, kc.y, __float_as_uint(__ldg(c.k_scale + so)), 0u);
            kv[i][1] = make_uint4(vc.x, vc.y, __float_as_uint(__ldg(c.v_scale + so)), 0u);
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const KvRow r = kv_row<LPR, RPT>(i, n, c.heads, c.hd);
        if (!r.live) continue;
        const int64_t out = (static_cast<int64_t>(r.token) * c.heads + r.head) * c.hd + r.col;
        if constexpr (Q8) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint4 q = kv[i][p];
                const float s = __uint_as_float(q.z);
                const float2 f0 = e4m3x2_f32(static_cast<uint16_t>(q.x)), f1 = e4m3x2_f32(static_cast<uint16_t>(q.x >> 16));
                const float2 f2 = e4m3x2_f32(static_cast<uint16_t>(q.y)), f3 = e4m3x2_f32(static_cast<uint16_t>(q.y >> 16));
                const float x[8] = {f0.x * s, f0.y * s, f1.x * s, f1.y * s, f2.x * s, f2.y * s, f3.x * s, f3.y * s};
                kv[i][p] = pack16(x, static_cast<__nv_bfloat16*>(nullptr));
            }
        }
        st_stream16(k_out + out, kv[i][0]);
        st_stream16(v_out + out, kv[i][1]);
    }
}

// Units of kKvThreads / lpr tokens of one head: what a block takes at a time.
inline long long kv_units(int n, int heads, int lpr)
{
    const long long per = kKvThreads / lpr;
    return (n + per - 1) / per * heads;
}

// One unit a block: with two or four the larger threads cost more occupancy than they gained (16001 tokens of 8 heads of
// 128 into e4m3: 18.2 us with one, 19.8 with two, 20.4 with four).
template <int LPR>
twell_status run_append(const KvView& c, const void* k, const void* v, int64_t ldk, int64_t ldv, const int32_t* slots,
                        int n, int32_t* status, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    auto kern = c.q8 ? kv_append_kernel<LPR, true> : kv_append_kernel<LPR, false>;
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>(kv_units(n, c.heads, LPR))), dim3(kKvThreads), 0, s, c,
                                  static_cast<const bf*>(k), static_cast<const bf*>(v), ldk, ldv, slots, n, status);
}

template <int LPR>
twell_status run_gather(const KvView& c, const int32_t* slots, int n, void* k_out, void* v_out, int32_t* status,
                        cudaStream_t s)
{
    using bf = __nv_bfloat16;
    const long long units = kv_units(n, c.heads, LPR);
    // several units a block once that still gives every SM several blocks (30011 tokens of 8 heads of 128 from e4m3: 33.6 us
    // with one, 30.0 with four)
    twell_host::DevInfo dev;
    if (twell_host::dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    const int rpt = units >= 4ll * kGatherRows * dev.sm_count ? kGatherRows : 1;
    auto kern = rpt == 1 ? (c.q8 ? kv_gather_kernel<LPR, true, 1> : kv_gather_kernel<LPR, false, 1>)
                         : (c.q8 ? kv_gather_kernel<LPR, true, kGatherRows> : kv_gather_kernel<LPR, false, kGatherRows>);
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>((units + rpt - 1) / rpt)), dim3(kKvThreads), 0, s, c, slots, n,
                                  static_cast<bf*>(k_out), static_cast<bf*>(v_out), status);
}

constexpr long long kMaxRows = 1ll << 30;  // rows (tokens x heads) of one call: indices stay in 32 bits

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
