// rope.cu -- position rotation of a step's new tokens: appending raw latent rows and indexer
// keys to the caches, and preparing the raw queries, with the rotation applied on the way.
//
// Pair i (i = 0..31) of the 64 rotated values at position p turns by the angle p * f_i:
//   a' = a cos(p f_i) - b sin(p f_i),   b' = a sin(p f_i) + b cos(p f_i)
// with (a, b) the values (2i, 2i + 1) (interleaved) or (i, i + 32) (halves).
//
// Angles.  p f_i reaches a million radians, where an fp32 product is off by 0.03 rad and fp32
// range reduction cannot mend it.  Each warp lane owns one pair and turns its frequency into a
// 64-bit fraction of a full turn, step = f_i / (2 pi) * 2^64 (double arithmetic, once per warp);
// p * step in wrapping 64-bit integer arithmetic is then the angle modulo one turn, exactly, to
// p * 2^-64 turns.  sincospif of its top 32 bits, less the nearest quarter turn, gives cos and sin to 1e-7.
//
// Both kernels move bytes and little else (about 10 operations a rotated pair): a warp owns one
// token (append) or one head of one row (queries) and every long access is 16 bytes a lane.
// Measured: 4,000 rows of queries 249 us (5.1 TB/s); 32,768 tokens into FP8 entries 24.8 us (2.9 TB/s), 2,500 into bf16
// rows 2 us in a graph.  The FP8 append is bound by latency more than by its 450 instructions a token: schedulers issue
// in 0.62 of their cycles, with 8.7 warps each, which wait for memory in 5.6 of the 14 cycles between two
// of their instructions; no pipe is busy for more than 0.4 of the time.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr float kE4m3Max = 448.0f;
// Warps per CTA, a token or a head each: four pack the SM's registers better than eight (append of 32,768
// tokens 24.6 instead of 26.5 us when it was measured, queries the same).
constexpr int kWarps = 4;

// The frequency as a fraction of a turn per position, in units of 2^-64 turns.  The product with
// 1/(2 pi) is carried in two doubles: one alone is off by 2^-55 turns, which a million positions
// would raise to 2^-35.
__device__ __forceinline__ unsigned long long turn_step(float f) {
    const double kInvTwoPiHi = 0.15915494309189535, kInvTwoPiLo = -9.839338337591243e-18;
    const double p = (double)f * kInvTwoPiHi;
    const double e = fma((double)f, kInvTwoPiHi, -p) + (double)f * kInvTwoPiLo;
    const double frac = p - rint(p);  // [-1/2, 1/2], exact (from floor(p) up, a small negative p would lose its bits)
    return (unsigned long long)__double2ll_rn(frac * 18446744073709551616.0) +
           (unsigned long long)__double2ll_rn(e * 18446744073709551616.0);
}

// The nearest quarter turn is taken off in integers: what is left, at most an eighth of a turn, is off by 2^-27 half
// turns (2.3e-8 rad) in fp32, where a value next to half a turn would be off by four times that.  With one unit in the
// last place of sincospif (6e-8 below 1) cos and sin are good to 9e-8.
__device__ __forceinline__ void cos_sin(float f, int pos, float& c, float& s) {
    const unsigned long long phase = turn_step(f) * (unsigned long long)(long long)pos;
    const unsigned top = (unsigned)(phase >> 32), quarter = (top + (1u << 29)) >> 30;
    float x, y;
    sincospif((float)(int)(top - (quarter << 30)) * 4.656612873077393e-10f, &y, &x);  // in half turns
    c = (quarter & 1) ? y : x;
    s = (quarter & 1) ? x : y;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = a * c - b * s, y = a * s + b * c;
    a = x;
    b = y;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

// Groups below this magnitude are stored as zeros: 1 / s of a smaller scale may overflow, and the residuals below may
// lose bits.  (Dividing there instead costs every append of 32,768 tokens 26.4 instead of 24.8 us.)
constexpr float kTiny = 8.271806125530277e-25f;  // 2^-80

// A group's scale amax / 448 (1 when all is zero or tiny) and its reciprocal, for x / scale of many x: with
// q = x r, r = 1 / s rounded to nearest, the residual x - q s is exact in a fused multiply-add and
// q + (x - q s) r is x / s rounded to nearest (Markstein, IBM J. Res. Dev. 34, 1990): three instructions for
// two values, where a division takes a dozen each.
// The codes are therefore those of a true division, bit for bit (but -0 comes out as 0).
struct GroupScale {
    float s;
    uint64_t s2, r2;  // -s and 1 / s, twice
    __device__ __forceinline__ explicit GroupScale(float amax) {
        s = amax >= kTiny ? amax / kE4m3Max : 1.f;
        const float r = 1.f / s;
        s2 = pack_f32x2(-s, -s);
        r2 = pack_f32x2(r, r);
    }
    // two e4m3 codes of x / s and y / s, rounded to nearest even, saturated to the finite range
    __device__ __forceinline__ uint32_t codes2(float x, float y) const {
        const uint64_t v = pack_f32x2(x, y);
        const uint64_t q = fma_f32x2(v, r2, 0);
        float a, b;
        unpack_f32x2(fma_f32x2(fma_f32x2(q, s2, v), r2, q), a, b);
        return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
};

// one value of a row of T
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// the warp's rope pair (a, b) of a 64-value row
template <typename T>
__device__ __forceinline__ float2 load_pair(const T* x, int lane, int pairs) {
    const int i = pairs == kRopeHalves ? lane : 2 * lane, j = pairs == kRopeHalves ? lane + 32 : 2 * lane + 1;
    return make_float2(load1(x + i), load1(x + j));
}
__device__ __forceinline__ void store_pair_bf16(__nv_bfloat16* x, int lane, int pairs, float2 v) {
    if (pairs == kRopeHalves) {
        x[lane] = __float2bfloat16_rn(v.x);
        x[lane + 32] = __float2bfloat16_rn(v.y);
    } else {
        reinterpret_cast<uint32_t*>(x)[lane] = pack_bf16(v.x, v.y);
    }
}

// A raw indexer row of d values (64 or 128): the lane's rotated pair and, of a wide row, two of the rest.
struct IndexRow {
    float2 v, w;
};
template <typename T>
__device__ __forceinline__ IndexRow load_index_row(const T* x, int d, int lane, int pairs) {
    IndexRow r;
    r.v = load_pair(x, lane, pairs);
    r.w = d == 128 ? make_float2(load1(x + 64 + 2 * lane), load1(x + 65 + 2 * lane)) : make_float2(0.f, 0.f);
    return r;
}
// Turns its first 64 values and stores e4m3 codes and the row's scale (GroupScale), or
// fp32 values (scale == nullptr).  One warp.
__device__ __forceinline__ void store_index_row(IndexRow r, int d, int lane, int pairs, float c, float s, void* dst,
                                                float* scale) {
    if (pairs != kRopeNone) turn(r.v.x, r.v.y, c, s);
    const int i = pairs == kRopeHalves ? lane : 2 * lane, j = pairs == kRopeHalves ? lane + 32 : 2 * lane + 1;
    if (scale == nullptr) {
        float* o = reinterpret_cast<float*>(dst);
        o[i] = r.v.x;
        o[j] = r.v.y;
        if (d == 128) reinterpret_cast<float2*>(o + 64)[lane] = r.w;
        return;
    }
    const float m = warp_max(fmaxf(fmaxf(fabsf(r.v.x), fabsf(r.v.y)), fmaxf(fabsf(r.w.x), fabsf(r.w.y))));
    const GroupScale sc(m);
    uint8_t* o = reinterpret_cast<uint8_t*>(dst);
    const uint32_t cv = sc.codes2(r.v.x, r.v.y);
    if (pairs == kRopeHalves) {
        o[i] = (uint8_t)cv;
        o[j] = (uint8_t)(cv >> 8);
    } else {
        reinterpret_cast<uint16_t*>(o)[lane] = (uint16_t)cv;
    }
    if (d == 128) reinterpret_cast<uint16_t*>(o + 64)[lane] = (uint16_t)sc.codes2(r.w.x, r.w.y);
    if (lane == 0) *scale = sc.s;
}

__global__ void __launch_bounds__(32 * kWarps) append_rope_kernel(const RopeAppendArgs a) {
    const int i = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= a.n) return;
    // every load that needs no other goes out at once (the values are dropped where the token is bad)
    const int b = __ldg(a.seq + i), s = __ldg(a.pos + i);
    const float f = __ldg(a.inv_freq + lane);
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.kv_new) + (int64_t)i * a.kv_stride;
    const uint4 l0 = __ldcs(reinterpret_cast<const uint4*>(v) + lane);
    const uint4 l1 = __ldcs(reinterpret_cast<const uint4*>(v) + 32 + lane);
    float2 r = load_pair(v + kDV, lane, a.latent_pairs);
    const IndexRow key =
        a.k_bf16 ? load_index_row(reinterpret_cast<const __nv_bfloat16*>(a.k_new) + (int64_t)i * a.k_stride, a.d_I, lane,
                                  a.index_pairs)
                 : load_index_row(reinterpret_cast<const float*>(a.k_new) + (int64_t)i * a.k_stride, a.d_I, lane,
                                  a.index_pairs);
    if (b < 0 || b >= a.B || s < 0 || s >= a.T_max) {
        if (lane == 0) record_status(a.status, DSA_STATUS_LENGTH);
        return;
    }
    int64_t row = (int64_t)b * a.T_max + s;
    int pb = 0;
    if (a.block_table != nullptr) pb = __ldg(a.block_table + (int64_t)b * a.max_blocks + (s >> a.block_shift));
    float c, sn;
    cos_sin(f, s, c, sn);
    if (a.latent_pairs != kRopeNone) turn(r.x, r.y, c, sn);
    if (a.block_table != nullptr) {
        if (pb < 0 || pb >= a.num_blocks) {
            if (lane == 0) record_status(a.status, DSA_STATUS_INDEX_OOB);
            return;
        }
        row = ((int64_t)pb << a.block_shift) + (s & ((1 << a.block_shift) - 1));
    }

    // ---- latent row
    if (!a.kv_fp8) {
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.kv) + row * kDK;
        reinterpret_cast<uint4*>(dst)[lane] = l0;
        reinterpret_cast<uint4*>(dst)[32 + lane] = l1;
        store_pair_bf16(dst + kDV, lane, a.latent_pairs, r);
    } else {
        // lanes 0..15 of load h hold group 2h of 128 values, lanes 16..31 group 2h + 1
        uint8_t* e = reinterpret_cast<uint8_t*>(a.kv) + row * kFp8EntryBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 u = h ? l1 : l0;
            const float2 x[4] = {unpack_bf16(u.x), unpack_bf16(u.y), unpack_bf16(u.z), unpack_bf16(u.w)};
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const GroupScale sc(m);
            uint2 w;
            w.x = sc.codes2(x[0].x, x[0].y) | (sc.codes2(x[1].x, x[1].y) << 16);
            w.y = sc.codes2(x[2].x, x[2].y) | (sc.codes2(x[3].x, x[3].y) << 16);
            reinterpret_cast<uint2*>(e + 256 * h)[lane] = w;
            if ((lane & 15) == 0) reinterpret_cast<float*>(e + kFp8ScaleOff)[2 * h + (lane >> 4)] = sc.s;
        }
        store_pair_bf16(reinterpret_cast<__nv_bfloat16*>(e + kFp8RopeOff), lane, a.latent_pairs, r);
    }

    // ---- indexer key
    void* kd = reinterpret_cast<uint8_t*>(a.k_I) + row * a.d_I * (a.idx_fp8 ? 1 : 4);
    float* ks = a.idx_fp8 ? a.k_scale + row : nullptr;
    store_index_row(key, a.d_I, lane, a.index_pairs, c, sn, kd, ks);
}

// A warp has one head of a row; blockIdx.y counts groups of kWarps MLA heads first, then of indexer heads.
// (Several heads a warp, with cos and sin made once and loads ahead, were slower: what counts here is how many
// warps' loads are in flight. 4,000 rows, us: one head 254, two 254, four 273, a loop over a third of the row 259 to 297.)
__global__ void __launch_bounds__(32 * kWarps) rope_queries_kernel(const RopeQueryArgs a) {
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float f = __ldg(a.inv_freq + lane);
    const int pos = __ldg(a.pos + t);
    float c, sn;
    if ((int)blockIdx.y < a.mla_groups) {
        const int h = blockIdx.y * kWarps + warp;
        if (h >= a.H) return;
        const int64_t th = (int64_t)t * a.H + h;
        float2 r = load_pair(reinterpret_cast<const __nv_bfloat16*>(a.q_pe) + (int64_t)t * a.pe_row_stride +
                                 (int64_t)h * a.pe_head_stride,
                             lane, a.latent_pairs);
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.q) + th * kDK);
        if (a.q_nope != nullptr) {
            const uint4* src = reinterpret_cast<const uint4*>(a.q_nope) + th * (kDV / 8);
            const uint4 l0 = __ldg(src + lane), l1 = __ldg(src + 32 + lane);
            dst[lane] = l0;
            dst[32 + lane] = l1;
        }
        cos_sin(f, pos, c, sn);
        if (a.latent_pairs != kRopeNone) turn(r.x, r.y, c, sn);
        store_pair_bf16(reinterpret_cast<__nv_bfloat16*>(dst) + kDV, lane, a.latent_pairs, r);
        return;
    }
    const int h = (blockIdx.y - a.mla_groups) * kWarps + warp;
    if (h >= a.H_I) return;
    const int64_t th = (int64_t)t * a.H_I + h, off = (int64_t)t * a.qi_row_stride + (int64_t)h * a.d_I;
    const IndexRow x =
        a.qi_bf16 ? load_index_row(reinterpret_cast<const __nv_bfloat16*>(a.qi_new) + off, a.d_I, lane, a.index_pairs)
                  : load_index_row(reinterpret_cast<const float*>(a.qi_new) + off, a.d_I, lane, a.index_pairs);
    cos_sin(f, pos, c, sn);
    store_index_row(x, a.d_I, lane, a.index_pairs, c, sn, reinterpret_cast<uint8_t*>(a.q_I) + th * a.d_I * (a.idx_fp8 ? 1 : 4),
                    a.idx_fp8 ? a.q_scale + th : nullptr);
}

}  // namespace

cudaError_t launch_append_rope(const RopeAppendArgs& a, cudaStream_t st) {
    if (a.n == 0) return cudaSuccess;
    append_rope_kernel<<<(a.n + kWarps - 1) / kWarps, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_rope_queries(RopeQueryArgs a, cudaStream_t st) {
    a.mla_groups = a.q_pe != nullptr ? (a.H + kWarps - 1) / kWarps : 0;
    const int groups = a.mla_groups + (a.qi_new != nullptr ? (a.H_I + kWarps - 1) / kWarps : 0);
    if (a.Nq == 0 || groups == 0) return cudaSuccess;
    rope_queries_kernel<<<dim3(a.Nq, groups), 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dsa
