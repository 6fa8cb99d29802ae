// twell_rope.cu -- rotary positions: each pair of a head's values turned by an angle that its token's position gives.
//
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),  t = position x frequency of the pair;  backward: -t
//
// Bounded by memory traffic where tokens are many (every value read and written once) and by the launch where they are
// few. A thread keeps the turns of V pairs of one token in registers and takes them through the heads, so that an angle is
// formed once a token where tokens fill the device. 16001 tokens of 24 heads of 128 in bf16 34.0 us, 86% of the copy rate (what
// is left: 68 registers a thread leave 38% of the warps, too few loads under way); 16384 in fp32 61.1 us, 97%; one token 1.75.
// The angle is formed in integers: a frequency is a count of 2^-64 turns a position, so that position x frequency modulo
// 2^64 is the fraction of a turn, whatever the position (an fp32 product is off by 0.06 rad a million positions away). The
// upper 32 bits are cut into a quarter of a turn and a rest within +-1/8, whose sine and cosine are their power series.
#include "twell_common.cuh"
#include "twell_mma.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeThreads = 32 * kRopeWarps;
// Heads a thread has under way at a time (16001 tokens of 24 heads of 128 in bf16: 33.6 us with two, 34.2 with four, whose
// registers cost warps; without any in advance 35.0).
constexpr int kRopeHeads = 2;
constexpr int kRopeMaxDim = 1024;

struct RopeSide {
    const void* in;
    void* out;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;  // elements
};
struct RopeArgs {
    RopeSide q, k;
    const int32_t* positions;
    const uint64_t* turns;
    int64_t pos_batch;
    int q_heads, heads;  // heads: of q and k together
    int tokens, S, hd, rot;
    int pair_chunks, chunks;  // of a head: V pairs each, then those that are copied, 2 V elements each
    int lanes;                // warps that share a chunk's heads: kRopeWarps of each of so many blocks
    unsigned unit_blocks;
    float cos_factor, sin_factor;
};

template <typename E, int V>
struct alignas(V * sizeof(E)) RopeVec {
    E v[V];
};
template <typename E, int V>
__device__ __forceinline__ void rope_unpack(const RopeVec<E, V>& x, float* o)
{
    if constexpr (sizeof(E) == 2 && V > 1) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = Elem<E>::to_f(x.v[i]);
    }
}
template <typename E, int V>
__device__ __forceinline__ void rope_pack(const float* o, RopeVec<E, V>& x)
{
    if constexpr (sizeof(E) == 2 && V > 1) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = bf16x2_rn(o[2 * i], o[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x.v[i] = Elem<E>::from_f(o[i]);
    }
}

// cos and sin of position x frequency. The rest r of the turn after the nearest quarter is at most pi / 4 in radians:
// the series end at r^9 / 9! and r^10 / 10!, off by 2e-9 and 1e-10. What the rounding of r to fp32 adds is 2^-24 of it.
__device__ __forceinline__ void rope_turn(int32_t position, uint64_t turns, float& c, float& s)
{
    const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns + 0x80000000ull;
    const uint32_t f = static_cast<uint32_t>(p >> 32);
    const uint32_t quarter = (f + 0x20000000u) >> 30;
    const float r = static_cast<float>(static_cast<int32_t>(f - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    const float r2 = r * r;
    const float sr = r + r * r2 * fmaf(r2, fmaf(r2, fmaf(r2, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f);
    const float cr = fmaf(
        r2, fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, -1.0f / 3628800.0f, 1.0f / 40320.0f), -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
    const float x = (quarter & 1) ? sr : cr, y = (quarter & 1) ? cr : sr;
    c = (quarter + 1) & 2 ? -x : x;
    s = quarter & 2 ? -y : y;
}

// NEIGHBOURS: a pair is (2i, 2i + 1), else (i, i + rot / 2). Either way a chunk of V pairs is two vectors of V elements. A block
// has 32 chunks (of one token after the other), each warp of it every lanes-th head of them.
template <typename E, int V, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a)
{
    using Vec = RopeVec<E, V>;
    __shared__ float2 turn[V][32];
    pdl_begin();
    const unsigned u = blockIdx.x % a.unit_blocks * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
    const int lane = static_cast<int>(blockIdx.x / a.unit_blocks * kRopeWarps + warp);
    const int tok = static_cast<int>(u / static_cast<unsigned>(a.chunks)), chunk = static_cast<int>(u - tok * a.chunks);
    const bool live = tok < a.tokens;
    const int b = a.S == a.tokens ? 0 : tok / a.S, t = tok - b * a.S;
    const bool turned = chunk < a.pair_chunks;
    // where the chunk's two vectors begin in a head; the second of the last copied chunk may lie past it
    const int lo = turned ? chunk * (NEIGHBOURS ? 2 * V : V) : a.rot + (chunk - a.pair_chunks) * 2 * V;
    const int hi = turned && !NEIGHBOURS ? lo + a.rot / 2 : lo + V;
    const bool both = hi < a.hd;
    // the queries' heads from `lane` on, then the keys', which go on where those ended, so that the lanes have as many
    bool keys = lane >= a.q_heads;
    int h = keys ? lane - a.q_heads : lane;
    const E* in;
    E* out;
    auto enter = [&](const RopeSide& s) {
        in = static_cast<const E*>(s.in) + b * s.in_batch + t * s.in_token + lo;
        out = static_cast<E*>(s.out) + b * s.out_batch + t * s.out_token + lo;
    };
    enter(keys ? a.k : a.q);
    Vec x[kRopeHeads][2];
    // heads first, first + lanes, ... of a side that has `count` of them, `stride` apart
    auto request = [&](int first, int count, int64_t stride) {
#pragma unroll
        for (int i = 0; i < kRopeHeads; ++i)
            if (first + i * a.lanes < count) {
                const E* p = in + (first + i * a.lanes) * stride;
                x[i][0] = *reinterpret_cast<const Vec*>(p);
                if (both) x[i][1] = *reinterpret_cast<const Vec*>(p + (hi - lo));
            }
    };
    int heads = keys ? a.heads - a.q_heads : a.q_heads;
    if (live) request(h, heads, keys ? a.k.in_head : a.q.in_head);
    // the warps share a chunk's angles out between them
    if (live && turned) {
        const int32_t pos = __ldg(a.positions + b * a.pos_batch + t);
#pragma unroll
        for (int i = 0; i < (V + kRopeWarps - 1) / kRopeWarps; ++i) {
            const int pair = i * kRopeWarps + static_cast<int>(warp);
            if (pair < V) {
                float2 cs;
                rope_turn(pos, __ldg(a.turns + chunk * V + pair), cs.x, cs.y);
                turn[pair][threadIdx.x & 31] = make_float2(cs.x * a.cos_factor, cs.y * a.sin_factor);
            }
        }
    }
    __syncthreads();
    if (!live) return;
    // (cos, cos), (sin, sin) and (-sin, -sin) of two pairs each
    constexpr int kTwos = (V + 1) / 2;
    F2 c[kTwos], sn[kTwos], ns[kTwos];
#pragma unroll
    for (int j = 0; j < kTwos; ++j) {
        const float2 p = turned ? turn[2 * j][threadIdx.x & 31] : make_float2(1.0f, 0.0f);
        const float2 q = turned && V > 1 ? turn[(2 * j + 1) % V][threadIdx.x & 31] : p;
        c[j] = F2::of(p.x, q.x);
        sn[j] = F2::of(p.y, q.y);
        ns[j] = F2::of(-p.y, -q.y);
    }
    auto finish = [&](int first, int count, int64_t stride) {
#pragma unroll
        for (int i = 0; i < kRopeHeads; ++i) {
            if (first + i * a.lanes >= count) break;
            if (turned) {
                float v[2 * V];
                rope_unpack<E, V>(x[i][0], v);
                rope_unpack<E, V>(x[i][1], v + V);
#pragma unroll
                for (int j = 0; j < kTwos; ++j) {
                    // the first values of pairs 2j and 2j + 1 are v[e] and v[f], their second ones kStep behind
                    constexpr int kStep = NEIGHBOURS ? 1 : V;
                    const int e = NEIGHBOURS ? 4 * j : 2 * j, f = V == 1 ? e : NEIGHBOURS ? e + 2 : e + 1;
                    const F2 m = F2::of(v[e], v[f]), w = F2::of(v[e + kStep], v[f + kStep]);
                    fma2(w, ns[j], m * c[j]).get(v[e], v[f]);
                    fma2(w, c[j], m * sn[j]).get(v[e + kStep], v[f + kStep]);
                }
                rope_pack<E, V>(v, x[i][0]);
                rope_pack<E, V>(v + V, x[i][1]);
            }
            E* p = out + (first + i * a.lanes) * stride;
            *reinterpret_cast<Vec*>(p) = x[i][0];
            if (both) *reinterpret_cast<Vec*>(p + (hi - lo)) = x[i][1];
        }
    };
    const int step = kRopeHeads * a.lanes;
    bool here = true;  // the heads from h on are requested
    for (;;) {
        for (; h < heads; h += step) {
            if (!here) request(h, heads, keys ? a.k.in_head : a.q.in_head);
            here = false;
            finish(h, heads, keys ? a.k.out_head : a.q.out_head);
        }
        if (keys || a.q_heads == a.heads) return;
        keys = true;
        heads = a.heads - a.q_heads;
        h = (lane + a.lanes - a.q_heads % a.lanes) % a.lanes;
        enter(a.k);
    }
}

// Elements of a vector that every address of the call allows: a power of two up to 16 bytes.
int vector_of(const RopeArgs& a, bool has_k, int elem, bool copies)
{
    int v = 16 / elem;
    auto fits = [&](int64_t n) { return n % v == 0; };
    auto side = [&](const RopeSide& s, int heads) {
        const int64_t bytes = static_cast<int64_t>(v) * elem;
        return reinterpret_cast<uintptr_t>(s.in) % bytes == 0 && reinterpret_cast<uintptr_t>(s.out) % bytes == 0 &&
               (a.tokens == a.S || (fits(s.in_batch) && fits(s.out_batch))) &&
               (a.S == 1 || (fits(s.in_token) && fits(s.out_token))) && (heads == 1 || (fits(s.in_head) && fits(s.out_head)));
    };
    // rot / 2 pairs in vectors of V: the same condition for both layouts
    while (v > 1 && !(fits(a.rot / 2) && (!copies || fits(a.hd - a.rot)) && side(a.q, a.q_heads) &&
                      (!has_k || side(a.k, a.heads - a.q_heads))))
        v /= 2;
    return v;
}

template <typename E, int V>
twell_status launch_rope(const RopeArgs& a, bool neighbours, unsigned blocks, cudaStream_t s)
{
    return twell_host::launch_dep(neighbours ? rope_kernel<E, V, true> : rope_kernel<E, V, false>, dim3(blocks),
                                  dim3(kRopeThreads), 0, s, a);
}

// Whether the tokens' heads of an output lie apart: each axis in turn, from the smallest stride on, steps past what the
// axes before it span.
bool apart(const int64_t (&stride)[3], const int64_t (&size)[3], int64_t hd)
{
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[order[j]] < stride[order[i]]) {
                const int o = order[i];
                order[i] = order[j];
                order[j] = o;
            }
    int64_t span = hd;
    for (int i : order) {
        if (size[i] == 1) continue;
        if (stride[i] < span) return false;
        span += (size[i] - 1) * stride[i];
    }
    return true;
}

}  // namespace
}  // namespace twell

using namespace twell_host;

namespace {

bool rope_side(const twell_rope_heads* h, int32_t B, int32_t S, int32_t hd, int elem, twell::RopeSide* out)
{
    if (h->in == nullptr || h->out == nullptr || reinterpret_cast<uintptr_t>(h->in) % elem != 0 ||
        reinterpret_cast<uintptr_t>(h->out) % elem != 0)
        return false;
    const int64_t in[3] = {h->in_batch, h->in_token, h->in_head}, to[3] = {h->out_batch, h->out_token, h->out_head};
    const int64_t size[3] = {B, S, h->n_heads};
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 1) continue;
        if (in[i] < 0 || in[i] > INT64_MAX / size[i] / 8 || to[i] > INT64_MAX / size[i] / 8) return false;
        if (h->in == h->out && in[i] != to[i]) return false;
    }
    if (!twell::apart(to, size, hd)) return false;
    *out = twell::RopeSide{h->in, h->out, in[0], in[1], in[2], to[0], to[1], to[2]};
    return true;
}

twell_status rope(const twell_rope_heads* q, const twell_rope_heads* k, const int32_t* positions, int64_t pos_batch,
                  const uint64_t* turns, float factor, int32_t B, int32_t S, int32_t hd, int32_t rot, int32_t neighbours,
                  twell_dtype dtype, bool backward, void* stream)
{
    if (q == nullptr || B < 0 || S < 0 || hd <= 0 || rot <= 0 || rot % 2 != 0 || rot > hd || q->n_heads <= 0 ||
        (k != nullptr && k->n_heads <= 0) || (neighbours != 0 && neighbours != 1) || !(factor > 0.0f) || factor > 3.0e38f)
        return TWELL_ERR_INVALID;
    if (!dtype_ok(dtype) || hd > twell::kRopeMaxDim) return TWELL_ERR_UNSUPPORTED;
    if (B == 0 || S == 0) return TWELL_OK;
    const int elem = dtype == TWELL_BF16 ? 2 : 4;
    twell::RopeArgs a = {};
    if (positions == nullptr || turns == nullptr || reinterpret_cast<uintptr_t>(positions) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(turns) % 8 != 0 || pos_batch < 0 || !rope_side(q, B, S, hd, elem, &a.q) ||
        (k != nullptr && (!rope_side(k, B, S, hd, elem, &a.k) || k->out == q->out || k->out == q->in || q->out == k->in)))
        return TWELL_ERR_INVALID;
    const long long tokens = static_cast<long long>(B) * S, heads = static_cast<long long>(q->n_heads) + (k ? k->n_heads : 0);
    if (tokens * hd > INT32_MAX || heads > 65535) return TWELL_ERR_UNSUPPORTED;
    a.positions = positions;
    a.turns = turns;
    a.pos_batch = pos_batch;
    a.q_heads = q->n_heads;
    a.heads = static_cast<int>(heads);
    a.tokens = static_cast<int>(tokens);
    a.S = S;
    a.hd = hd;
    a.rot = rot;
    a.cos_factor = factor;
    a.sin_factor = backward ? -factor : factor;
    // in place the rest of a head stays where it is
    const bool copies = rot < hd && (q->in != q->out || (k != nullptr && k->in != k->out));
    const int v = twell::vector_of(a, k != nullptr, elem, copies);
    a.pair_chunks = rot / 2 / v;
    a.chunks = a.pair_chunks + (copies ? (hd - rot + 2 * v - 1) / (2 * v) : 0);
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    const long long units = (tokens * a.chunks + 31) / 32, want = 16ll * dev.sm_count, most = (heads + twell::kRopeWarps - 1) / twell::kRopeWarps;
    const long long groups = units >= want ? 1 : (want + units - 1) / units < most ? (want + units - 1) / units : most;
    a.lanes = static_cast<int>(groups) * twell::kRopeWarps;
    a.unit_blocks = static_cast<unsigned>(units);
    const unsigned blocks = static_cast<unsigned>(units * groups);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool nb = neighbours != 0;
    if (dtype == TWELL_BF16) {
        using bf = __nv_bfloat16;
        return v == 8   ? twell::launch_rope<bf, 8>(a, nb, blocks, s)
               : v == 4 ? twell::launch_rope<bf, 4>(a, nb, blocks, s)
               : v == 2 ? twell::launch_rope<bf, 2>(a, nb, blocks, s)
                        : twell::launch_rope<bf, 1>(a, nb, blocks, s);
    }
    return v == 4   ? twell::launch_rope<float, 4>(a, nb, blocks, s)
           : v == 2 ? twell::launch_rope<float, 2>(a, nb, blocks, s)
                    : twell::launch_rope<float, 1>(a, nb, blocks, s);
}

}  // namespace

extern "C" twell_status twell_rope_fwd(const twell_rope_heads* q, const twell_rope_heads* k, const int32_t* positions,
                                       int64_t pos_batch, const uint64_t* turns, float factor, int32_t B, int32_t S,
                                       int32_t head_dim, int32_t rot_dim, int32_t neighbours, twell_dtype dtype, void* stream)
{
    return rope(q, k, positions, pos_batch, turns, factor, B, S, head_dim, rot_dim, neighbours, dtype, false, stream);
}

extern "C" twell_status twell_rope_bwd(const twell_rope_heads* dq, const twell_rope_heads* dk, const int32_t* positions,
                                       int64_t pos_batch, const uint64_t* turns, float factor, int32_t B, int32_t S,
                                       int32_t head_dim, int32_t rot_dim, int32_t neighbours, twell_dtype dtype, void* stream)
{
    return rope(dq, dk, positions, pos_batch, turns, factor, B, S, head_dim, rot_dim, neighbours, dtype, true, stream);
}
