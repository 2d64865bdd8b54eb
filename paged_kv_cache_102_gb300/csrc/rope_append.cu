// Rotary positions of queries and keys, and the appends that go with them:
// rotated keys and values into a 16-bit cache, an E4M3 cache with one scale,
// or an E4M3 cache with a scale for each (block, kv head).
//
// Rotation of the pair (a, b) of channels at position pos with inverse
// frequency w:  (a cos - b sin, b cos + a sin),  cos, sin of pos * w times a
// factor.  Pairs are channels (i, i + R/2) or, interleaved, (2i, 2i + 1);
// channels from R = rotary_dim on pass unchanged.
//
// Angles: pos * w reaches 10^6 radians and more, where a binary32 product has
// lost the angle.  The kernel works in turns: w / 2pi becomes a 64-bit
// fixed-point fraction of a turn (error below 2^-64, from the exact product
// of w's 24-bit mantissa and 2^66 / 2pi rounded to an integer), and the
// 64-bit product with pos wraps around exactly as the angle does, so the
// phase is right to pos * 2^-64 turns at every position.  The nearest quarter
// turn is split off in integers and sincospi runs on the rest.
//
// Block scales: a "run" is a maximal stretch of consecutive tokens of the call
// with consecutive slots of one block.  For a run at offset o of its block and
// one kv head, K and V alike:
//   need = the least power of two 2^e, -64 <= e <= 120, with max|x| <= 448 * 2^e
//   new  = o == 0 ? need : max(old, need)
// the run's elements are stored as e4m3(x / new), and where new > old the
// block's other codes are requantised as e4m3(code * (old / new)).  Scales are
// powers of two because a block fills over many calls: when a later token
// raises the scale, the old codes move by a power of two, which loses nothing
// but what falls among the subnormal codes, however often it happens.  (An
// E4M3 code has the same relative precision at every exponent, so a scale that
// is not a power of two would gain nothing.)  Non-finite elements do not enter
// the maximum: an infinity saturates to 448 * new, a NaN stays a NaN code.
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kWindow = 32;  // tokens whose runs one warp looks over at a time
constexpr int kScaleMinExp = -64, kScaleMaxExp = 120;

// w / 2pi as a 64-bit fraction of a turn.
__device__ __forceinline__ uint64_t turn_of(float w) {
    const uint32_t bits = __float_as_uint(w);
    const int be = (bits >> 23) & 0xff;
    const uint64_t m = (bits & 0x7fffffu) | (be ? 0x800000u : 0u);
    const uint64_t c = 11743562013128004906ull;  // 2^66 / 2pi, to the nearest integer
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    const int s = 2 - ((be ? be : 1) - 150);  // w = m * 2^(be - 150), phase = (m c) >> s
    uint64_t t;
    if (s >= 128) t = 0;
    else if (s >= 64) t = hi >> (s - 64);
    else if (s > 0) t = (lo >> s) | (hi << (64 - s));
    else t = s > -64 ? lo << -s : 0;
    return (bits >> 31) ? 0 - t : t;
}

// cos and sin of a phase in 64-bit turns.
__device__ __forceinline__ void cos_sin_turns(uint64_t phase, float& c, float& s) {
    const uint64_t q = (phase + (1ull << 61)) >> 62;  // nearest quarter turn
    const int64_t r = static_cast<int64_t>(phase - (q << 62));
    float s0, c0;
    sincospif(__ll2float_rn(r) * 0x1p-63f, &s0, &c0);  // r * 2^-63 half turns, at most 1/4
    const bool odd = q & 1;
    const float cc = odd ? s0 : c0, ss = odd ? c0 : s0;
    c = (q == 1 || q == 2) ? -cc : cc;
    s = (q & 2) ? -ss : ss;
}

// The eight channels 8c .. 8c+7 of a row, as this lane holds them: their
// frequencies, and cos and sin at one position.
struct RopeLane {
    uint64_t turn[8];
    float cs[8], sn[8];

    __device__ __forceinline__ void frequencies(const RopeAppendParams& p, int c) {
        const int half = p.rotary_dim / 2;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 8 * c + j;
            if (p.interleaved && (j & 1)) {
                turn[j] = turn[j - 1];
                continue;
            }
            const int i = p.interleaved ? e / 2 : (e < half ? e : e - half);
            turn[j] = e < p.rotary_dim ? turn_of(p.inv_freq[i]) : 0;
        }
    }
    __device__ __forceinline__ void at(const RopeAppendParams& p, int pos, int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (p.interleaved && (j & 1)) {
                cs[j] = cs[j - 1];
                sn[j] = sn[j - 1];
            } else if (8 * c + j < p.rotary_dim) {
                cos_sin_turns(turn[j] * static_cast<uint64_t>(static_cast<int64_t>(pos)), cs[j], sn[j]);
                cs[j] *= p.factor;
                sn[j] *= p.factor;
            } else {
                cs[j] = 1.f;
                sn[j] = 0.f;
            }
        }
    }
};

template <int ACT>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
    Vec16<ACT>::to_float(u, f);
}

template <int ACT>
__device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = static_cast<uint32_t>(float_to_act<ACT>(f[2 * i])) |
               (static_cast<uint32_t>(float_to_act<ACT>(f[2 * i + 1])) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rotate the eight channels x of chunk c (raw bits u) in place.  Every lane of
// the warp calls it: the partner chunk of the half layout comes from the lane
// that holds it when R/2 is a multiple of 8, from memory otherwise.  Products
// and their difference are rounded one by one (no fused multiply-add), which
// keeps the result symmetric in the two terms.
template <int ACT>
__device__ __forceinline__ void rotate8(const RopeAppendParams& p, const RopeLane& rl, const uint4& u,
                                        const uint16_t* row, int c, int lane, bool live, float* x) {
    const int rot = p.rotary_dim, half = rot / 2;
    float y[8];
    if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
    } else if (half % 8 == 0) {
        const int hc = half / 8;
        const int src = c < hc ? lane + hc : (c < 2 * hc ? lane - hc : lane);
        uint4 v;
        v.x = __shfl_sync(0xffffffffu, u.x, src);
        v.y = __shfl_sync(0xffffffffu, u.y, src);
        v.z = __shfl_sync(0xffffffffu, u.z, src);
        v.w = __shfl_sync(0xffffffffu, u.w, src);
        unpack<ACT>(v, y);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 8 * c + j;
            y[j] = live && e < rot ? act_to_float<ACT>(row[e < half ? e + half : e - half]) : 0.f;
        }
        __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = 8 * c + j;
        if (e >= rot) continue;
        const bool first = p.interleaved ? !(j & 1) : e < half;
        const float a = __fmul_rn(x[j], rl.cs[j]), b = __fmul_rn(y[j], rl.sn[j]);
        x[j] = first ? __fsub_rn(a, b) : __fadd_rn(a, b);
    }
}

__device__ __forceinline__ uint2 to_codes(const float* x) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = a | (b << 16);
    }
    return make_uint2(w[0], w[1]);
}

// x / s: the product with an exact reciprocal when s is a power of two within
// 2^-126 .. 2^126 (the same value, without a division), else the quotient.
__device__ __forceinline__ void divide8(float* x, float s) {
    const uint32_t b = __float_as_uint(s), e = b >> 23;
    if ((b & 0x7fffffu) == 0 && e >= 1 && e <= 253) {
        const float r = __uint_as_float((254u - e) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], s);
    }
}

// Token t's slot: -1 for padding (negative slot or position) and for a slot
// outside the pool (*bad is set).
__device__ __forceinline__ int64_t slot_of(const RopeAppendParams& p, int t, bool* bad) {
    if (t < 0 || t >= p.num_tokens) return -1;
    const int64_t s = p.slot_mapping[t];
    if (s < 0 || (p.positions && p.positions[t] < 0)) return -1;
    if (s >= static_cast<int64_t>(p.num_blocks) * p.block_size) {
        *bad = true;
        return -1;
    }
    return s;
}

// ---------------------------------------------------------------------------
// Rows that do not share a scale: the queries and, for a 16-bit or
// one-scale E4M3 cache, the keys and values.  The rows of a token are its
// heads [q | k | v]; one warp takes rows [part * per, (part + 1) * per) of a
// token, RP = 32 / (D / 8) of them at a time, so that cos and sin are computed
// once for all of them.
// ---------------------------------------------------------------------------
template <int ACT, int CACHE>
__device__ __forceinline__ void plain_rows(const RopeAppendParams& p, int token, int row0, int row1) {
    const int lane = threadIdx.x & 31;
    const int lpr = p.head_dim / 8, rp = 32 / lpr;
    const int r = lane / lpr, c = lane - r * lpr;
    const int pos = p.positions[token];
    if (pos < 0) return;  // padding: q_out keeps its row
    bool bad = false;
    const int64_t slot = slot_of(p, token, &bad);
    if (bad && row0 == 0 && lane == 0) atomicOr(p.err, kErrBadSlot);
    int64_t blk = 0;
    int off = 0;
    if (slot >= 0) divmod_u(slot, p.block_size, blk, off);
    RopeLane rl;
    rl.frequencies(p, c);
    rl.at(p, pos, c);
    for (int h0 = row0; h0 < row1; h0 += rp) {
        const int h = h0 + r;
        const bool have = r < rp && h < row1;
        const bool is_q = h < p.num_q_heads, is_k = !is_q && h < p.num_q_heads + p.num_kv_heads;
        const int hk = is_q ? h : is_k ? h - p.num_q_heads : h - p.num_q_heads - p.num_kv_heads;
        const uint16_t* src = is_q   ? static_cast<const uint16_t*>(p.q) + token * p.q_stride
                              : is_k ? static_cast<const uint16_t*>(p.k) + token * p.k_stride
                                     : static_cast<const uint16_t*>(p.v) + token * p.v_stride;
        src += static_cast<int64_t>(hk) * p.head_dim;
        const uint4 u = have ? *reinterpret_cast<const uint4*>(src + c * 8) : make_uint4(0u, 0u, 0u, 0u);
        float x[8];
        unpack<ACT>(u, x);
        rotate8<ACT>(p, rl, u, src, c, lane, have && (is_q || is_k), x);
        if (!have) continue;
        if (is_q) {
            uint16_t* dst = static_cast<uint16_t*>(p.q_out) + token * p.q_out_stride + static_cast<int64_t>(h) * p.head_dim;
            *reinterpret_cast<uint4*>(dst + c * 8) = 8 * c < p.rotary_dim ? pack<ACT>(x) : u;
            continue;
        }
        if (slot < 0) continue;
        const int64_t dst = ((blk * p.num_kv_heads + hk) * p.block_size + off) * p.head_dim + c * 8;
        if constexpr (CACHE == ACT) {
            uint16_t* cache = static_cast<uint16_t*>(is_k ? p.k_cache : p.v_cache);
            *reinterpret_cast<uint4*>(cache + dst) = is_k && 8 * c < p.rotary_dim ? pack<ACT>(x) : u;
        } else {
            if (!is_k) unpack<ACT>(u, x);
            divide8(x, is_k ? *p.k_scale : *p.v_scale);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + dst) = to_codes(x);
        }
    }
}

// ---------------------------------------------------------------------------
// One run of tokens of one block and kv head into a block-scaled cache, K or
// V, by one warp: the maximum over the run, the block's new scale, its other
// codes where the scale grew, the run's codes.
// ---------------------------------------------------------------------------
template <int ACT>
__device__ __forceinline__ void scaled_run(const RopeAppendParams& p, int t0, int64_t slot0, int head, bool is_k) {
    const int lane = threadIdx.x & 31;
    const int lpr = p.head_dim / 8, rp = 32 / lpr;
    const int r = lane / lpr, c = lane - r * lpr;
    int64_t blk;
    int off0;
    divmod_u(slot0, p.block_size, blk, off0);
    // length: up to the end of the block
    const int most = p.block_size - off0;
    int n = 1;
    for (int base = 1; base < most; base += 32) {
        const int k = base + lane;
        bool bad = false;
        const bool in = k < most && slot_of(p, t0 + k, &bad) == slot0 + k;
        const unsigned out = __ballot_sync(0xffffffffu, !in);
        n = base + (out ? __ffs(out) - 1 : 32);
        if (out) break;
    }
    const bool turn = is_k && p.positions != nullptr;
    const uint16_t* src0 = is_k ? static_cast<const uint16_t*>(p.k) + t0 * p.k_stride
                                : static_cast<const uint16_t*>(p.v) + t0 * p.v_stride;
    src0 += static_cast<int64_t>(head) * p.head_dim;
    const int64_t stride = is_k ? p.k_stride : p.v_stride;
    RopeLane rl;
    if (turn) rl.frequencies(p, c);
    auto load = [&](int i, float* x) {  // row i of the run (every lane calls it)
        const bool have = r < rp && i < n;
        const uint16_t* src = src0 + (have ? i : 0) * stride;
        const uint4 u = have ? *reinterpret_cast<const uint4*>(src + c * 8) : make_uint4(0u, 0u, 0u, 0u);
        unpack<ACT>(u, x);
        if (turn) {
            rl.at(p, have ? p.positions[t0 + i] : 0, c);
            rotate8<ACT>(p, rl, u, src, c, lane, have, x);
        }
        return have;
    };
    float top = 0.f;
    for (int i0 = 0; i0 < n; i0 += rp) {
        float x[8];
        load(i0 + r, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = fabsf(x[j]);
            if (a <= 3.402823466e38f) top = fmaxf(top, a);  // false for NaN and infinity
        }
    }
    top = warp_max(top);
    // top = 1.m * 2^e: 448 = 1.75 * 2^8
    int e = kScaleMinExp;
    if (top > 0.f) {
        const uint32_t b = __float_as_uint(top);
        e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = min(kScaleMaxExp, max(kScaleMinExp, e));
    }
    const float need = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    float* scale = (is_k ? p.k_scales : p.v_scales) + blk * p.num_kv_heads + head;
    const float old = off0 == 0 ? 0.f : *scale;
    const float now = old > need ? old : need;  // a scale that is not positive counts as none
    uint8_t* tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) +
                    (blk * p.num_kv_heads + head) * p.block_size * p.head_dim;
    if (now != old) {
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *scale = now;
        if (old > 0.f) {
            const float ratio = __fdiv_rn(old, now);
            for (int i = lane; i < p.block_size * lpr; i += 32) {
                const int row = i / lpr;
                if (row >= off0 && row < off0 + n) continue;
                uint2* at = reinterpret_cast<uint2*>(tile) + i;
                const uint2 codes = *at;
                float x[16];
                Vec16E4M3::to_float(make_uint4(codes.x, codes.y, 0u, 0u), x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= ratio;
                *at = to_codes(x);
            }
        }
    }
    for (int i0 = 0; i0 < n; i0 += rp) {
        float x[8];
        const int i = i0 + r;
        if (!load(i, x)) continue;
        divide8(x, now);
        *reinterpret_cast<uint2*>(tile + (off0 + i) * p.head_dim + c * 8) = to_codes(x);
    }
}

// Grid: the first kv_ctas * kv_windows blocks (block-scaled cache only) take
// the runs that start in a window of kWindow tokens, kv_ctas blocks a window;
// the others take (token, part of its rows) items, one a warp.
template <int ACT, int CACHE>
__global__ void __launch_bounds__(kWarps * 32)
    rope_append_kernel(const RopeAppendParams p, int kv_windows, int kv_ctas, int parts, int per, int rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int cta = blockIdx.x;
    if constexpr (CACHE == kE4M3B) {
        if (cta < kv_windows * kv_ctas) {
            const int w = cta / kv_ctas;
            const int t = w * kWindow + lane;
            bool bad = false, unused = false;
            const int64_t slot = slot_of(p, t, &bad);
            const int64_t prev = slot_of(p, t - 1, &unused);
            if (bad && warp == 0 && cta == w * kv_ctas) atomicOr(p.err, kErrBadSlot);
            bool first = slot >= 0;
            if (first && prev == slot - 1) {
                int64_t blk;
                int off;
                divmod_u(slot, p.block_size, blk, off);
                first = off == 0;
            }
            const unsigned leaders = __ballot_sync(0xffffffffu, first);
            const int items = __popc(leaders) * p.num_kv_heads * 2;
            for (int it = (cta - w * kv_ctas) * kWarps + warp; it < items; it += kv_ctas * kWarps) {
                const int run = it / (p.num_kv_heads * 2), hv = it - run * p.num_kv_heads * 2;
                const int at = __fns(leaders, 0, run + 1);
                scaled_run<ACT>(p, w * kWindow + at, __shfl_sync(0xffffffffu, slot, at), hv >> 1, !(hv & 1));
            }
            return;
        }
        cta -= kv_windows * kv_ctas;
    }
    const int64_t item = static_cast<int64_t>(cta) * kWarps + warp;
    const int token = static_cast<int>(item / parts);
    if (token >= p.num_tokens) return;
    const int row0 = static_cast<int>(item - static_cast<int64_t>(token) * parts) * per;
    plain_rows<ACT, CACHE>(p, token, row0, min(rows, row0 + per));
}

template <int ACT, int CACHE>
cudaError_t launch(const RopeAppendParams& p, cudaStream_t stream) {
    const int rp = 32 / (p.head_dim / 8);
    int kv_windows = 0, kv_ctas = 0;
    if (CACHE == kE4M3B) {
        kv_windows = (p.num_tokens + kWindow - 1) / kWindow;
        // few windows (a decode step): one warp an item, every token a run
        const int64_t items = static_cast<int64_t>(kWindow) * p.num_kv_heads * 2;
        const int64_t want = 152 * 8 / kv_windows + 1;
        const int64_t most = (items + kWarps - 1) / kWarps;
        kv_ctas = static_cast<int>(want < most ? want : most);
    }
    const int rows = p.positions == nullptr ? 0 : CACHE == kE4M3B ? p.num_q_heads : p.num_q_heads + 2 * p.num_kv_heads;
    // rows of a token per warp: all of them when the tokens alone fill the GPU
    const int passes = (rows + rp - 1) / rp;
    int split = 1;
    while (split < passes && static_cast<int64_t>(p.num_tokens) * split < 152 * 16) split *= 2;
    const int per = rows ? (passes + split - 1) / split * rp : 1;
    const int parts = rows ? (rows + per - 1) / per : 0;
    const int64_t plain = (static_cast<int64_t>(p.num_tokens) * parts + kWarps - 1) / kWarps;
    const int64_t grid = static_cast<int64_t>(kv_windows) * kv_ctas + plain;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    rope_append_kernel<ACT, CACHE><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(
        p, kv_windows, kv_ctas, parts > 0 ? parts : 1, per, rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int act, int cache, cudaStream_t s) {
    if (act == kF16)
        return cache == kF16     ? launch<kF16, kF16>(p, s)
               : cache == kE4M3  ? launch<kF16, kE4M3>(p, s)
               : cache == kE4M3B ? launch<kF16, kE4M3B>(p, s)
                                 : cudaErrorInvalidValue;
    return cache == kBF16    ? launch<kBF16, kBF16>(p, s)
           : cache == kE4M3  ? launch<kBF16, kE4M3>(p, s)
           : cache == kE4M3B ? launch<kBF16, kE4M3B>(p, s)
                             : cudaErrorInvalidValue;
}

}  // namespace pkv
