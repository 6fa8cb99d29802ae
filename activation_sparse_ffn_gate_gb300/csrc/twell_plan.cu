// twell_plan.cu -- a served step's plan, made on the device: pages for the requests' new tokens from a ring of free ones, the
// pages of requests that have ended back into it, and slot, position and owner of each of the step's tokens.
//
// Three sums over the requests say everything: of the new tokens (where a request's tokens lie in the step), of the pages
// taken (which page of the ring is whose) and of the pages given back. Every block forms them for itself, in shared memory
// (4096 requests are 32 KB to read, from L2 but for the first), and then does its share of the tokens and pages, each of
// which finds its request by bisection. Pages are taken at the ring's head and given back behind its last free page, so that
// within a call nothing is written that the call still reads, and the result does not depend on any order.
// Bounded by the launch and a chain of loads (state and lengths, then pages) for a decode step, by the 12 bytes a token that
// it writes for long prompts: 16 requests 2.4 us, 500 with pieces of prompts and ended ones among them 4.0, 924000 tokens of 37
// prompts 7.2 (11 MB, which stay in L2).
#include "twell_common.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kPlanMaxSeqs = 4096;
constexpr int kPlanWarpPer = 4;  // requests a lane where one warp has all of them
constexpr int kPlanBlocks = 8;   // most blocks an SM
constexpr int kEnded = -1;

struct PlanArgs {
    int32_t* ring;
    int32_t* state;  // the ring's first free page, the number of free ones, a count that is zero between calls
    int32_t* table;
    const int32_t* lens;
    const int32_t* news;
    const int32_t* labels;
    int32_t *slots, *positions, *owner, *starts, *lens_out, *state_out, *status;
    int n_pages, page_shift, max_pages, B, M;
};

// Sums of non-negative numbers that stop at 2^31 - 1.
__device__ __forceinline__ int sat_add(int a, int b)
{
    return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7fffffffu));
}

// The sums of two numbers over the lanes before this one and over all of them, in a warp.
__device__ __forceinline__ void warp_scan(int (&v)[2], int (&total)[2])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        int incl = v[e];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = sat_add(incl, u);
        }
        total[e] = __shfl_sync(0xffffffffu, incl, 31);
        const int before = __shfl_up_sync(0xffffffffu, incl, 1);
        v[e] = lane ? before : 0;
    }
}
// The same over the threads of a block. `red` has a place for each warp and number.
template <int THREADS>
__device__ __forceinline__ void block_scan(int (&v)[2], int (&red)[2][32], int (&total)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum[2];
    warp_scan(v, sum);
    if (lane < 2) red[lane][warp] = sum[lane];
    __syncthreads();
    int w[2] = {lane < THREADS / 32 ? red[0][lane] : 0, lane < THREADS / 32 ? red[1][lane] : 0};
    warp_scan(w, total);
#pragma unroll
    for (int e = 0; e < 2; ++e) v[e] = sat_add(v[e], __shfl_sync(0xffffffffu, w[e], warp));
    __syncthreads();
}

// The last i < n with at[i] <= v (at ascending, at[0] <= v).
__device__ __forceinline__ int last_at_most(const int* at, int n, int v)
{
    int lo = 0, len = n;
    while (len > 1) {
        const int half = len >> 1;
        if (at[lo + half] <= v) lo += half;
        len -= half;
    }
    return lo;
}

// What the sums come to: tokens, pages taken and given back, the ring before the step.
struct PlanSums {
    int tokens, taken, given, head, free;
};

// PER requests a thread of the block or, with WARP, of its first warp; Q adjacent tokens at a time.
template <int PER, int THREADS, bool WARP, int Q>
__global__ void __launch_bounds__(THREADS) kv_plan_kernel(const PlanArgs a)
{
    extern __shared__ int plan_smem[];
    __shared__ int red[2][32];
    __shared__ PlanSums s_sums;
    __shared__ int s_last;
    pdl_begin();
    int* start = plan_smem;          // [B + 1] of the requests' tokens in the step
    int* past = start + a.B + 1;     // [B] tokens that they had, -1 where they get none
    int* first = past + a.B;         // [B] of their pages among those taken
    int* back = first + a.B;         // [B] of their pages among those given back
    const int page = 1 << a.page_shift, tid = static_cast<int>(threadIdx.x);
    constexpr int kSpread = WARP ? 32 : THREADS;  // threads that have the requests
    const bool counts = !WARP || tid < 32;
    const int per = (a.B + kSpread - 1) / kSpread, b0 = tid * per;
    int had[PER], add[PER];  // a request: tokens it had, its new ones
    bool ends[PER], wrong[PER];
    if (counts) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool is = i < per && b0 + i < a.B;
            had[i] = is ? a.lens[b0 + i] : 0;
            add[i] = is ? a.news[b0 + i] : 0;
        }
        int head = a.state[0], free = a.state[1];
        if (!WARP && tid == 0) s_sums.taken = 0;
        bool bad = head < 0 || free < 0 || free > a.n_pages || (head >= a.n_pages && (head != 0 || free != 0));
        if (bad) head = free = 0;  // an empty ring: nothing is taken from it, and the pages of ended requests go to its cells from 0 on
        // a length rounded up to a page stays within 32 bits
        const long long cap = min(static_cast<long long>(a.max_pages) << a.page_shift, 0x7fffffffll - 1023);
        auto scan = [&](int (&v)[2], int (&total)[2]) {
            if constexpr (WARP) warp_scan(v, total);
            else block_scan<THREADS>(v, red, total);
        };
        int sum[2] = {0, 0}, total[2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int n = add[i];
            add[i] = max(n, 0);
            ends[i] = n == kEnded;
            wrong[i] = n < kEnded || had[i] < 0 || static_cast<long long>(had[i]) + add[i] > cap;
            sum[0] = sat_add(sum[0], add[i]);
        }
        scan(sum, total);
        const int tokens = total[0];
        int at = sum[0];
        // pages: a request whose tokens do not all have a place in the step or in its row of the table gets none
        int need[PER], gives[PER];
        sum[0] = sum[1] = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            need[i] = gives[i] = 0;
            if (i < per && b0 + i < a.B) {
                start[b0 + i] = at;
                if (add[i] > 0 && static_cast<long long>(at) + add[i] > a.M) wrong[i] = true;
                at = sat_add(at, add[i]);
                if (!wrong[i]) {
                    const int held = (had[i] + page - 1) >> a.page_shift;
                    if (ends[i]) gives[i] = held;
                    else if (add[i] > 0) need[i] = static_cast<int>((static_cast<long long>(had[i]) + add[i] + page - 1) >> a.page_shift) - held;
                }
                bad |= wrong[i];
                sum[0] = sat_add(sum[0], need[i]);
                sum[1] = sat_add(sum[1], gives[i]);
            }
        }
        scan(sum, total);
        int take = sum[0], give = sum[1], given = total[1];
        // more pages than there are: some are given back twice, and none are taken back
        const bool refuse = static_cast<long long>(free) + given > a.n_pages;
        if (refuse) given = 0;
        bad |= refuse;
        bool empty = false;
        int taken = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i < per && b0 + i < a.B) {
                const bool none = need[i] > 0 && sat_add(take, need[i]) > free;
                empty |= none;
                past[b0 + i] = wrong[i] || none ? -1 : had[i];
                first[b0 + i] = take;
                back[b0 + i] = give;
                take = sat_add(take, need[i]);
                if (need[i] > 0 && !none) taken = take;
                give = sat_add(give, gives[i]);
                if (wrong[i] || none) add[i] = 0;
                had[i] = ends[i] && !wrong[i] && !refuse ? 0 : had[i] + add[i];  // the length after the step
            }
        }
        taken = __reduce_max_sync(0xffffffffu, taken);
        if (WARP) {
            if (tid == 0) s_sums.taken = taken;
        } else if ((tid & 31) == 0 && taken > 0) {
            atomicMax(&s_sums.taken, taken);
        }
        if (tid == 0) {
            start[a.B] = s_sums.tokens = tokens;
            s_sums.given = given;
            s_sums.head = head;
            s_sums.free = free;
        }
        if (blockIdx.x == 0 && bad) report(a.status, TWELL_ERR_DEVICE_CHECK);
        if (blockIdx.x == 0 && empty) report(a.status, TWELL_ERR_POOL_EMPTY);
    }
    __syncthreads();
    const int tokens = s_sums.tokens, taken = s_sums.taken, given = s_sums.given, head = s_sums.head, free = s_sums.free;

    // lengths and state may be written where they were read once every block has read them: the last to say so does it
    const bool in_place = a.lens_out == a.lens || a.state_out == a.state;
    bool commit = blockIdx.x == 0;
    if (in_place && gridDim.x > 1) {
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(a.state + 2, 1) == static_cast<int>(gridDim.x) - 1;
        }
        __syncthreads();
        commit = s_last != 0;
    }
    if (commit) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (counts && i < per && b0 + i < a.B) a.lens_out[b0 + i] = had[i];
        for (int i = tid; i <= a.B; i += THREADS) a.starts[i] = start[i];
        if (tid == 0) {
            const long long h = static_cast<long long>(head) + taken;
            a.state_out[0] = static_cast<int>(h >= a.n_pages && a.n_pages > 0 ? h - a.n_pages : h);
            a.state_out[1] = free - taken + given;
            a.state_out[2] = a.state_out[3] = 0;
            if (in_place && gridDim.x > 1) a.state[2] = 0;
        }
    }

    auto ring_at = [&](int i) {  // the i-th cell from the head on, i < n_pages
        const long long j = static_cast<long long>(head) + i;
        return a.ring + (j >= a.n_pages ? j - a.n_pages : j);
    };
    auto row = [&](int b, int p) { return a.table + static_cast<long long>(b) * a.max_pages + p; };
    const unsigned threads = gridDim.x * THREADS, me = blockIdx.x * THREADS + tid;

    // tokens, Q at a time: where each one's page stands, the pages, the slots
    const unsigned groups = (static_cast<unsigned>(a.M) + Q - 1) / Q;
    for (unsigned u = me; u < groups; u += threads) {
        const int i0 = static_cast<int>(u * Q), end = min(tokens, a.M);
        int pos[Q], own[Q], pg[Q];
        bool live[Q], same[Q];  // has a place; is in the page of the one before
        const int32_t* from[Q];
        int b = a.B > 0 ? last_at_most(start, a.B, i0) : 0, page_of = -1;
#pragma unroll
        for (int e = 0; e < Q; ++e) {
            const int i = i0 + e;
            pos[e] = 0;
            own[e] = -1;
            live[e] = same[e] = false;
            from[e] = nullptr;
            if (i >= end) continue;
            while (i >= start[b + 1]) ++b, page_of = -1;
            own[e] = b;
            if (past[b] < 0) continue;
            live[e] = true;
            pos[e] = past[b] + (i - start[b]);
            const int p = pos[e] >> a.page_shift, held = (past[b] + page - 1) >> a.page_shift;
            same[e] = e > 0 && p == page_of;
            page_of = p;
            if (!same[e]) from[e] = p < held ? row(b, p) : ring_at(first[b] + p - held);
        }
#pragma unroll
        for (int e = 0; e < Q; ++e) {
            pg[e] = from[e] != nullptr ? *from[e] : -1;
            if (a.labels != nullptr && own[e] >= 0) own[e] = __ldg(a.labels + own[e]);
        }
        int slot[Q];
#pragma unroll
        for (int e = 0; e < Q; ++e) {
            if (same[e]) pg[e] = pg[e - (e > 0)];
            const bool is = live[e] && pg[e] >= 0 && pg[e] < a.n_pages;
            if (live[e] && !is) report(a.status, TWELL_ERR_DEVICE_CHECK);
            slot[e] = is ? (pg[e] << a.page_shift) + (pos[e] & (page - 1)) : -1;
        }
        if (Q % 4 == 0 && i0 + Q <= a.M) {
#pragma unroll
            for (int e = 0; e + 3 < Q; e += 4) {
                *reinterpret_cast<int4*>(a.slots + i0 + e) = make_int4(slot[e], slot[e + 1], slot[e + 2], slot[e + 3]);
                *reinterpret_cast<int4*>(a.positions + i0 + e) = make_int4(pos[e], pos[e + 1], pos[e + 2], pos[e + 3]);
                *reinterpret_cast<int4*>(a.owner + i0 + e) = make_int4(own[e], own[e + 1], own[e + 2], own[e + 3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < Q; ++e)
                if (i0 + e < a.M) {
                    a.slots[i0 + e] = slot[e];
                    a.positions[i0 + e] = pos[e];
                    a.owner[i0 + e] = own[e];
                }
        }
    }
    // pages taken, into the table; by the last threads first, since the first ones have tokens
    for (unsigned u = threads - 1 - me; u < static_cast<unsigned>(taken); u += threads) {
        const int j = static_cast<int>(u), b = last_at_most(first, a.B, j);
        *row(b, ((past[b] + page - 1) >> a.page_shift) + j - first[b]) = *ring_at(j);
    }
    // pages given back, behind the free ones
    for (unsigned u = threads - 1 - me; u < static_cast<unsigned>(given); u += threads) {
        const int j = static_cast<int>(u), b = last_at_most(back, a.B, j);
        const int pg = *row(b, j - back[b]);
        if (pg < 0 || pg >= a.n_pages) report(a.status, TWELL_ERR_DEVICE_CHECK);
        *ring_at(free + j) = pg;
    }
}

// The page of a token waits for the sums, so that a step is quickest with one token a thread, as far as one block an SM goes (16
// requests: 2.8 us, with four 4.1); beyond that a thread takes four, most of which share a page (924000 tokens: 7.3 us, 7.8 with
// eight, 18.8 with one).
template <int PER, int THREADS, bool WARP, int Q>
twell_status launch_plan(const PlanArgs& a, long long blocks, cudaStream_t s)
{
    auto kern = kv_plan_kernel<PER, THREADS, WARP, Q>;
    static std::atomic<uint64_t> allowed{0};
    constexpr size_t kMost = (4 * (WARP ? 32 * PER : PER * THREADS) + 1) * sizeof(int);
    if (twell_host::allow_smem(kern, kMost, allowed) != TWELL_OK) return TWELL_ERR_CUDA;
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>(std::max(blocks, 1ll))), dim3(THREADS),
                                  (4 * static_cast<size_t>(a.B) + 1) * sizeof(int), s, a);
}
template <int PER, int THREADS, bool WARP>
twell_status run_plan(const PlanArgs& a, int sms, cudaStream_t s)
{
    const long long ones = (static_cast<long long>(a.M) + THREADS - 1) / THREADS, most = static_cast<long long>(sms) * kPlanBlocks;
    if (ones <= sms) return launch_plan<PER, THREADS, WARP, 1>(a, ones, s);
    return launch_plan<PER, THREADS, WARP, 4>(a, std::min((ones + 3) / 4, most), s);
}

}  // namespace
}  // namespace twell

using namespace twell_host;

extern "C" twell_status twell_kv_plan(const twell_page_pool* pool, int32_t* page_table, int32_t max_pages,
                                      const int32_t* seq_lens, const int32_t* new_lens, const int32_t* labels, int32_t B,
                                      int32_t n_tokens, int32_t* slots, int32_t* positions, int32_t* owner, int32_t* starts,
                                      int32_t* seq_lens_out, int32_t* state_out, int32_t* dev_status, void* stream)
{
    if (pool == nullptr || pool->n_pages < 0 || pool->page_size <= 0 || max_pages <= 0 || B < 0 || n_tokens < 0)
        return TWELL_ERR_INVALID;
    if ((pool->page_size & (pool->page_size - 1)) != 0 || pool->page_size > 1024 || B > twell::kPlanMaxSeqs ||
        static_cast<long long>(pool->n_pages) * pool->page_size > INT32_MAX || n_tokens > INT32_MAX - 65536)
        return TWELL_ERR_UNSUPPORTED;
    const void* need[] = {pool->state, starts, state_out, dev_status};
    for (const void* p : need)
        if (p == nullptr) return TWELL_ERR_INVALID;
    if (pool->n_pages > 0 && pool->ring == nullptr) return TWELL_ERR_INVALID;
    if (B > 0 && (page_table == nullptr || seq_lens == nullptr || new_lens == nullptr || seq_lens_out == nullptr))
        return TWELL_ERR_INVALID;
    if (n_tokens > 0 && (slots == nullptr || positions == nullptr || owner == nullptr)) return TWELL_ERR_INVALID;
    if (!aligned16(slots) || !aligned16(positions) || !aligned16(owner)) return TWELL_ERR_INVALID;
    if (B > 0 && (seq_lens_out == new_lens || seq_lens_out == labels)) return TWELL_ERR_INVALID;  // read while it is written
    const void* words[] = {pool->ring, pool->state, page_table, seq_lens, new_lens, labels, starts, seq_lens_out, state_out};
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) % sizeof(int32_t) != 0) return TWELL_ERR_INVALID;
    int shift = 0;
    while ((1 << shift) < pool->page_size) ++shift;
    const twell::PlanArgs a = {pool->ring, pool->state, page_table,   seq_lens,  new_lens,   labels, slots, positions, owner,
                               starts,     seq_lens_out, state_out,   dev_status, pool->n_pages, shift, max_pages, B, n_tokens};
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B <= 32) return twell::run_plan<1, 256, true>(a, dev.sm_count, s);
    if (B <= 32 * twell::kPlanWarpPer) return twell::run_plan<twell::kPlanWarpPer, 256, true>(a, dev.sm_count, s);
    if (B <= 512) return twell::run_plan<1, 512, false>(a, dev.sm_count, s);
    return twell::run_plan<twell::kPlanMaxSeqs / 512, 512, false>(a, dev.sm_count, s);
}
