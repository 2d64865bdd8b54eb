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
// with consecutive slots of one block.  Runs of one block apply in the call's
// order (split_runs).  For a run at offset o of its block and
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
#include <type_traits>

#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kTable = 4096;  // floats of cos and sin a block keeps in shared memory
constexpr int kLoads = 4;     // row loads a warp has in flight where rows do not share a scale
constexpr int kFill = 152 * 4;  // blocks that keep the GPU busy
constexpr int kScaleMinExp = -64, kScaleMaxExp = 120;

// How the channels of a pair lie: neighbours; R/2 apart with R/2 a multiple of
// 8 (whole 8-channel chunks swap, by shuffle); R/2 apart otherwise (partners
// are read from memory).  kPairsNone: no rotation (the append alone).
enum : int { kPairsNext = 0, kPairsChunks = 1, kPairsApart = 2, kPairsNone = 3 };

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
__device__ __forceinline__ float2 cos_sin_turns(uint64_t phase) {
    const uint32_t q = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);  // nearest quarter turn
    // the rest, to 2^-32 turns (7e-10 of the pair's magnitude, a hundredth of binary32's rounding)
    const int r = static_cast<int>((static_cast<uint32_t>(phase >> 32) - (q << 30)));
    float s0, c0;
    sincospif(static_cast<float>(r) * 0x1p-31f, &s0, &c0);  // half turns, at most 1/4
    const bool odd = q & 1;
    const float cc = odd ? s0 : c0, ss = odd ? c0 : s0;
    return make_float2((q == 1 || q == 2) ? -cc : cc, (q & 2) ? -ss : ss);
}

__device__ __forceinline__ float2 cos_sin_at(const RopeAppendParams& p, int i, int pos) {
    const float2 cs = cos_sin_turns(turn_of(p.inv_freq[i]) * static_cast<uint64_t>(static_cast<int64_t>(pos)));
    return make_float2(cs.x * p.factor, cs.y * p.factor);
}

// The block's table: for each of its rows, cos of the pairs that a lane's chunk
// of 8 channels needs (J of them) in J / 4 quads, then sin, quad q of chunk c at
// float4 index (row * J / 2 + q) * C + c, so that the lanes of a quarter warp
// read 128 consecutive bytes.  Chunks c and c + C of the half layout share
// their pairs.
template <int PAIRS>
struct Table {
    static constexpr int J = PAIRS == kPairsNext ? 4 : 8;
    int C;  // chunks with entries
    __device__ __forceinline__ explicit Table(const RopeAppendParams& p)
        : C(PAIRS == kPairsChunks ? p.rotary_dim / 16 : (p.rotary_dim + 7) / 8) {}
    __device__ __forceinline__ int row_floats() const { return 2 * J * C; }
    // Pair of entry j of chunk c (past the end: any).
    __device__ __forceinline__ static int pair(const RopeAppendParams& p, int c, int j) {
        const int half = p.rotary_dim / 2;
        const int e = PAIRS == kPairsNext ? 4 * c + j : 8 * c + j;
        return PAIRS == kPairsApart ? (e < half ? e : min(e - half, half - 1)) : min(e, half - 1);
    }
    // All threads of the block: rows [0, rows) for tokens t0, t0 + 1, ...
    __device__ __forceinline__ void fill(const RopeAppendParams& p, float* table, int64_t t0, int rows) const {
        // a thread stays with one entry of a row (n <= 256 of them)
        const int n = J * C, teams = kWarps * 32 / n, team = threadIdx.x / n;
        const int k = threadIdx.x - team * n, c = k / J, j = k - c * J;
        if (team >= teams) return;
        const uint64_t turn = turn_of(p.inv_freq[pair(p, c, j)]);
        float* at = table + ((j >> 2) * C + c) * 4 + (j & 3);
        for (int row = team; row < rows; row += teams) {
            const float2 cs = cos_sin_turns(turn * static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + row])));
            at[row * 2 * n] = cs.x * p.factor;
            at[row * 2 * n + n] = cs.y * p.factor;
        }
    }
    // cos and sin of the 8 channels of chunk c; 1 and 0 for a chunk that does not turn.
    __device__ __forceinline__ void read(const RopeAppendParams& p, const float* table, int row, int c, float* cs,
                                         float* sn) const {
        if (8 * c >= p.rotary_dim) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cs[j] = 1.f;
                sn[j] = 0.f;
            }
            return;
        }
        const int cc = PAIRS == kPairsChunks && c >= C ? c - C : c;
        const float4* at = reinterpret_cast<const float4*>(table) + row * (J / 2) * C + cc;
#pragma unroll
        for (int q = 0; q < J / 4; ++q) {
            const float4 a = at[q * C], b = at[(J / 4 + q) * C];
            const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (PAIRS == kPairsNext) {
                    cs[2 * j] = cs[2 * j + 1] = ca[j];
                    sn[2 * j] = sn[2 * j + 1] = sa[j];
                } else {
                    cs[4 * q + j] = ca[j];
                    sn[4 * q + j] = sa[j];
                }
            }
        }
    }
    // The same without the table, for a row that it does not hold.
    __device__ __forceinline__ void compute(const RopeAppendParams& p, int pos, int c, float* cs, float* sn) const {
        const int cc = PAIRS == kPairsChunks && c >= C ? c - C : c;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 t = 8 * c < p.rotary_dim ? cos_sin_at(p, pair(p, cc, PAIRS == kPairsNext ? j / 2 : j), pos)
                                                  : make_float2(1.f, 0.f);
            cs[j] = t.x;
            sn[j] = t.y;
        }
    }
};

template <int ACT>
__device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (ACT == kBF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x = the rotated channels of chunk c (raw bits u of row `row`).  Every lane of
// the warp calls it.  The products and their sum are rounded one by one, so
// that both terms of a channel enter alike.  Half layout in whole chunks: the
// sign of the second term is put into the partner's bits, and a chunk that
// does not turn gets -0 for a partner (x * 1 + -0 * 0 is x, its sign too).
template <int ACT, int PAIRS>
__device__ __forceinline__ void rotate8(const RopeAppendParams& p, const uint4& u, const uint16_t* row, int c, int lane,
                                        bool live, const float* cs, const float* sn, float* x) {
    const int rot = p.rotary_dim, half = rot / 2;
    float y[8];
    Vec16<ACT>::to_float(u, x);
    if constexpr (PAIRS == kPairsChunks) {
        const int hc = half / 8;
        const bool turns = c < 2 * hc;
        const int src = c < hc ? lane + hc : (turns ? lane - hc : lane);
        const uint32_t keep = turns ? ~0u : 0u, flip = c < hc || !turns ? 0x80008000u : 0u;
        uint4 v;
        v.x = (__shfl_sync(0xffffffffu, u.x, src) & keep) ^ flip;
        v.y = (__shfl_sync(0xffffffffu, u.y, src) & keep) ^ flip;
        v.z = (__shfl_sync(0xffffffffu, u.z, src) & keep) ^ flip;
        v.w = (__shfl_sync(0xffffffffu, u.w, src) & keep) ^ flip;
        Vec16<ACT>::to_float(v, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(y[j], sn[j]));
        return;
    }
    if constexpr (PAIRS == kPairsNext) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (j & 1) ? x[j ^ 1] : -x[j ^ 1];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 8 * c + j;
            y[j] = live && e < rot ? act_to_float<ACT>(row[e < half ? e + half : e - half]) : 0.f;
            if (e < half) y[j] = -y[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(y[j], sn[j]));
        if (8 * c + j < rot) x[j] = a;
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

// Binary16 elements divided by 2^e stay in binary16: for -15 <= e <= 24 the
// factor is a binary16 value and the product exact, unless it falls among the
// subnormals, below 2^-14, where every E4M3 result is 0 (the least code is 2^-9).
// Half the instructions of the way through binary32.
__device__ __forceinline__ uint2 half_codes_of(const uint4& u, uint32_t factor2) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&w[i]), *reinterpret_cast<const __half2*>(&factor2));
        q[i] = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&y), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// Division by s: a product with the exact reciprocal when s is a power of two
// within 2^-126 .. 2^126 (the same value, without a division), else a quotient.
struct Divisor {
    float s, r;
    bool exact;
    __device__ __forceinline__ explicit Divisor(float scale) : s(scale) {
        const uint32_t b = __float_as_uint(s), e = b >> 23;
        exact = (b & 0x7fffffu) == 0 && e >= 1 && e <= 253;
        r = __uint_as_float((254u - e) << 23);
    }
    __device__ __forceinline__ bool half_exact() const { return exact && s >= 0x1p-15f && s <= 0x1p24f; }
    __device__ __forceinline__ uint2 half_codes(const uint4& u) const {
        const uint32_t h = __half_as_ushort(__float2half_rn(r));
        return half_codes_of(u, h | (h << 16));
    }
    __device__ __forceinline__ void divide8(float* x) const {
        if (exact) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= r;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], s);
        }
    }
};

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
// Rows that do not share a scale: the queries and, for a 16-bit or one-scale
// E4M3 cache, the keys and values.  A warp takes a range of one token's heads
// [q | k | v], RP = 32 / (D / 8) rows at a time and kLoads such loads ahead of
// their use, with the token's cos and sin in registers (read once from the
// block's table).  The memory bounds it: 57 us for prompts of 345 MB in 16 bits
// (90 % of what a copy reaches), 88 us for 590 MB of queries beside the scaled
// runs; a decode step, 6.2 us, its round trips.
// ---------------------------------------------------------------------------
template <int ACT, int CACHE, int PAIRS>
__device__ __forceinline__ void plain_rows(const RopeAppendParams& p, int token, int row0, int row1, const float* table, int table_row) {
    constexpr int U = kLoads;
    const int lane = threadIdx.x & 31;
    const int lpr = p.head_dim / 8, rp = 32 / lpr;
    const int r = lane / lpr, c = lane - r * lpr;
    bool bad = false;
    const int64_t slot = slot_of(p, token, &bad);
    if (CACHE != kE4M3B && bad && row0 == 0 && lane == 0) atomicOr(p.err, kErrBadSlot);
    int64_t blk = 0;
    int off = 0;
    if (CACHE != kE4M3B && slot >= 0) divmod_u(slot, p.block_size, blk, off);
    float cs[8], sn[8];
    Table<PAIRS>(p).read(p, table, table_row, c, cs, sn);
    const bool turns = 8 * c < p.rotary_dim;
    // heads [a, b) of one kind: src row, rotation or not, and where the result goes
    auto heads = [&](int a, int b, const uint16_t* src, auto turning, auto store) {
        for (int h0 = a; h0 < b; h0 += U * rp) {
            uint4 u[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = h0 + i * rp + r;
                u[i] = r < rp && h < b ? *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * p.head_dim + c * 8)
                                       : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (h0 + i * rp >= b) break;
                const int h = h0 + i * rp + r;
                const bool have = r < rp && h < b;
                float x[8];
                if constexpr (decltype(turning)::value) {
                    rotate8<ACT, PAIRS>(p, u[i], src + static_cast<int64_t>(h) * p.head_dim, c, lane, have, cs, sn, x);
                    if (PAIRS == kPairsApart) __syncwarp();  // in place: partners are read before they are written
                } else {
                    Vec16<ACT>::to_float(u[i], x);
                }
                if (have) store(h, u[i], x);
            }
        }
    };
    const int nq = p.num_q_heads, nk = p.num_kv_heads;
    if (row0 < nq) {
        uint16_t* out = static_cast<uint16_t*>(p.q_out) + token * p.q_out_stride + c * 8;
        heads(row0, min(row1, nq), static_cast<const uint16_t*>(p.q) + token * p.q_stride, std::true_type{},
              [&](int h, const uint4& u, const float* x) {
                  *reinterpret_cast<uint4*>(out + static_cast<int64_t>(h) * p.head_dim) = turns ? pack<ACT>(x) : u;
              });
    }
    if constexpr (CACHE != kE4M3B) {
        if (slot < 0) return;
        auto at = [&](int h) { return ((blk * nk + h) * p.block_size + off) * p.head_dim + c * 8; };
        auto put = [&](void* cache, const float* scale, bool raw, int h, const uint4& u, float* x) {
            if constexpr (CACHE == ACT) {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + at(h)) = raw ? u : pack<ACT>(x);
            } else {
                Divisor(*scale).divide8(x);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at(h)) = to_codes(x);
            }
        };
        const int k0 = max(row0 - nq, 0), k1 = min(row1 - nq, nk);
        if (k0 < k1)
            heads(k0, k1, static_cast<const uint16_t*>(p.k) + token * p.k_stride, std::true_type{},
                  [&](int h, const uint4& u, float* x) { put(p.k_cache, p.k_scale, !turns, h, u, x); });
        const int v0 = max(row0 - nq - nk, 0), v1 = row1 - nq - nk;
        if (v0 < v1)
            heads(v0, v1, static_cast<const uint16_t*>(p.v) + token * p.v_stride, std::false_type{},
                  [&](int h, const uint4& u, float* x) { put(p.v_cache, p.v_scale, true, h, u, x); });
    }
}

// The block's new scale (see the head of the file) for the run's largest
// element `top`, its old scale being `old` (0: starts afresh).
__device__ __forceinline__ float new_scale(float top, float old) {
    // top = 1.m * 2^e: 448 = 1.75 * 2^8
    int e = kScaleMinExp;
    if (top > 0.f) {
        const uint32_t b = __float_as_uint(top);
        e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = min(kScaleMaxExp, max(kScaleMinExp, e));
    }
    const float need = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    return old > need ? old : need;  // a scale that is not positive counts as none
}

// Codes of the block's rows outside [off0, off0 + n) times ratio, by `lanes`
// lanes of which this is number `first`; 8-byte pieces, loads ahead of stores.
// (A call: it is rare, and inlined it costs the common path registers.)
__device__ __noinline__ void requantise(uint8_t* tile, int rows, int lpr, int off0, int n, float ratio, int first,
                                           int lanes) {
    constexpr int B = 8;
    const int pieces = rows * lpr;
    uint2* at = reinterpret_cast<uint2*>(tile);
    for (int i0 = first; i0 < pieces; i0 += lanes * B) {
        uint2 codes[B];
        bool mine[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int i = i0 + lanes * k, row = i / lpr;
            mine[k] = i < pieces && (row < off0 || row >= off0 + n);
            codes[k] = mine[k] ? at[i] : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            float x[16];
            Vec16E4M3::to_float(make_uint4(codes[k].x, codes[k].y, 0u, 0u), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= ratio;
            if (mine[k]) at[i0 + lanes * k] = to_codes(x);
        }
    }
}

__device__ __forceinline__ void finite_top(const float* x, float& top) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = fabsf(x[j]);
        if (a <= 3.402823466e38f) top = fmaxf(top, a);  // false for NaN and infinity
    }
}

// Where a run goes and comes from, for one head and K or V.
struct RunRows {
    const uint16_t* src;  // first row
    int64_t stride;
    float* scale;
    uint8_t* tile;  // the block's codes
    const int32_t* positions;  // of the run's tokens; null: no rotation
};

// Row i of a run in chunk c of this lane as floats, rotated if it turns (every
// lane of the warp calls it).
template <int ACT, int PAIRS>
__device__ __forceinline__ void run_row(const RopeAppendParams& p, const RunRows& run, int i, int c, bool have, float* x) {
    const uint16_t* row = run.src + (have ? i : 0) * run.stride;
    const uint4 u = have ? *reinterpret_cast<const uint4*>(row + c * 8) : make_uint4(0u, 0u, 0u, 0u);
    if (PAIRS != kPairsNone && run.positions) {
        float cs[8], sn[8];
        Table<PAIRS>(p).compute(p, run.positions[have ? i : 0], c, cs, sn);
        rotate8<ACT, PAIRS>(p, u, row, c, threadIdx.x & 31, have, cs, sn, x);
    } else {
        Vec16<ACT>::to_float(u, x);
    }
}

// The largest finite element of the rows r, r + rp, ... of a run (one warp's).
// For runs that do not fit the registers: longer blocks, and in calls of up to about
// 1,200 tokens (scaled_step_kernel) every run of more than a pass.
template <int ACT, int PAIRS>
__device__ __noinline__ float run_top(const RopeAppendParams& p, const RunRows run, int n, int r, int rp, int c, bool idle) {
    float top = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += rp) {
        float x[8];
        run_row<ACT, PAIRS>(p, run, i0 + r, c, !idle && i0 + r < n, x);
        finite_top(x, top);
    }
    return warp_max(top);
}

template <int ACT, int PAIRS>
__device__ __noinline__ void run_codes(const RopeAppendParams& p, const RunRows run, int n, int off0, int r, int rp, int c,
                                       bool idle, float now) {
    const Divisor by(now);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += rp) {
        float x[8];
        const bool have = !idle && i0 + r < n;
        run_row<ACT, PAIRS>(p, run, i0 + r, c, have, x);
        by.divide8(x);
        if (have) *reinterpret_cast<uint2*>(run.tile + (off0 + i0 + r) * p.head_dim + c * 8) = to_codes(x);
    }
}

// ---------------------------------------------------------------------------
// One run of n tokens of one block and kv head into a block-scaled cache, K
// (TURN: rotated) or V, by W warps (one, or two that take every other pass and
// meet for the maximum): the maximum over the run, the block's new scale, its
// other codes where the scale grew, the run's codes.  A run of up to GROUP
// passes stays in registers between the maximum and the codes (rotated, if it
// turns, with cos and sin from the table's rows); a longer one is read twice.
// ---------------------------------------------------------------------------
template <int ACT, int PAIRS, int GROUP, int W, bool TURN>
__device__ __forceinline__ void scaled_run(const RopeAppendParams& p, const RunRows& run, int n, int off0, int lane_row,
                                           int c, const float* table, float* tops2) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lpr = p.head_dim / 8, rows = 32 / lpr;  // rows of a warp's pass
    const int rp = W * rows;                          // rows of a pass of all W warps
    const bool idle = lane_row >= rows;
    const int r = (W == 2 ? (warp & 1) * rows : 0) + lane_row;
    const float old = off0 == 0 ? 0.f : *run.scale;
    const bool fits = n <= GROUP * rp;
    // the pair's maximum; behind its barrier both warps have read the old scale
    auto joined_top = [&](float top) {
        if constexpr (W == 2) {
            if (lane == 0) tops2[warp] = top;
            asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
            top = fmaxf(top, tops2[warp ^ 1]);
        }
        return top;
    };
    float now;
    if (fits) {
        uint4 u[GROUP];
        float x[TURN ? GROUP : 1][8];
        float top = 0.f;
        const uint16_t* src = run.src + r * run.stride + c * 8;
        const int64_t src_step = rp * run.stride;
        const int left = idle ? 0 : n - r;  // this lane has pass j where j * rp < left
#pragma unroll
        for (int j = 0; j < GROUP; ++j, src += src_step)
            u[j] = j * rp < left ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
        [[maybe_unused]] uint32_t tops = 0;
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
            if (j * rp >= n) break;
            if constexpr (TURN) {
                const int i = j * rp + r;
                const bool have = !idle && i < n;
                float cs[8], sn[8];
                Table<PAIRS>(p).read(p, table, have ? i : 0, c, cs, sn);
                rotate8<ACT, PAIRS>(p, u[j], run.src + (have ? i : 0) * run.stride, c, lane, have, cs, sn, x[j]);
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[j][k]));
            } else {
                top_pairs<ACT>(u[j], tops);
            }
        }
        if (!TURN)
            top = fmaxf(act_to_float<ACT>(static_cast<uint16_t>(tops)), act_to_float<ACT>(static_cast<uint16_t>(tops >> 16)));
        top = warp_max(top);
        if (!(top <= 3.402823466e38f)) {  // an infinity among them: the largest finite one instead
            top = 0.f;
#pragma unroll
            for (int j = 0; j < GROUP; ++j) {
                if (j * rp >= n) break;
                float y[8];
                if constexpr (TURN) {
                    finite_top(x[j], top);
                } else {
                    Vec16<ACT>::to_float(u[j], y);
                    finite_top(y, top);
                }
            }
            top = warp_max(top);
        }
        now = new_scale(joined_top(top), old);
        const Divisor by(now);
        uint8_t* dst = run.tile + (off0 + r) * p.head_dim + c * 8;
        const int dst_step = rp * p.head_dim;
        if (ACT == kF16 && !TURN && by.half_exact()) {
#pragma unroll
            for (int j = 0; j < GROUP; ++j, dst += dst_step) {
                if (j * rp >= n) break;
                if (j * rp < left) *reinterpret_cast<uint2*>(dst) = by.half_codes(u[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < GROUP; ++j, dst += dst_step) {
                if (j * rp >= n) break;
                float y[8];
                if constexpr (TURN) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = x[j][k];
                } else {
                    Vec16<ACT>::to_float(u[j], y);
                }
                by.divide8(y);
                if (j * rp < left) *reinterpret_cast<uint2*>(dst) = to_codes(y);
            }
        }
    } else {
        now = new_scale(joined_top(run_top<ACT, PAIRS>(p, run, n, r, rp, c, idle)), old);
        run_codes<ACT, PAIRS>(p, run, n, off0, r, rp, c, idle, now);
    }
    if (now != old) {
        __syncwarp();  // every lane has read the old scale
        if (lane == 0 && (W == 1 || !(warp & 1))) *run.scale = now;
        // the block's other rows (last, when nothing else needs registers)
        if (old > 0.f)
            requantise(run.tile, p.block_size, lpr, off0, n, __fdiv_rn(old, now), W == 2 ? (warp & 1) * 32 + lane : lane,
                       32 * W);
    }
}

// The same for a run of one token (a decode step), where a row takes lpr lanes
// (a power of two): a warp takes 32 / lpr (head, K or V) items from item0 on.
template <int ACT, int PAIRS>
__device__ __forceinline__ void single_rows(const RopeAppendParams& p, int t0, int64_t blk, int off0, int item0,
                                            const float* table) {
    const int lane = threadIdx.x & 31;
    const int lpr = p.head_dim / 8;
    const int r = lane / lpr, c = lane - r * lpr;
    const int it = item0 + r;
    const bool have = it < 2 * p.num_kv_heads, is_k = it < p.num_kv_heads;
    const int head = !have ? 0 : is_k ? it : it - p.num_kv_heads;
    float* scale = (is_k ? p.k_scales : p.v_scales) + blk * p.num_kv_heads + head;
    const float old = off0 == 0 || !have ? 0.f : *scale;
    const uint16_t* src = (is_k ? static_cast<const uint16_t*>(p.k) + t0 * p.k_stride
                                : static_cast<const uint16_t*>(p.v) + t0 * p.v_stride) +
                          static_cast<int64_t>(head) * p.head_dim;
    const uint4 u = have ? *reinterpret_cast<const uint4*>(src + c * 8) : make_uint4(0u, 0u, 0u, 0u);
    float x[8];
    if constexpr (PAIRS != kPairsNone) {
        float cs[8], sn[8];
        Table<PAIRS>(p).read(p, table, 0, c, cs, sn);
        rotate8<ACT, PAIRS>(p, u, src, c, lane, have && is_k, cs, sn, x);
        if (!is_k) Vec16<ACT>::to_float(u, x);
    } else {
        Vec16<ACT>::to_float(u, x);
    }
    float top = 0.f;
    finite_top(x, top);
    for (int off = lpr / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (!have) return;
    const float now = new_scale(top, old);
    uint8_t* tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) +
                    (blk * p.num_kv_heads + head) * p.block_size * p.head_dim;
    Divisor(now).divide8(x);
    *reinterpret_cast<uint2*>(tile + off0 * p.head_dim + c * 8) = to_codes(x);
    if (now != old) {
        if (c == 0) *scale = now;  // (every lane read the old one before the shuffles)
        if (old > 0.f) requantise(tile, p.block_size, lpr, off0, 1, __fdiv_rn(old, now), c, lpr);
    }
}

// ---------------------------------------------------------------------------
// Blocks whose tokens are not one run: skipped tokens between them, slots left
// out, out of order or twice.  Their runs apply one after the other, in the
// call's order, by the warps that have the first one; at most kReach - 1 skipped
// tokens lie before a later one, and a token at offset 0 starts afresh.  The
// common path only asks small functions about them (prompts, whose registers are
// short: only sees that there may be such a run) and leaves as the last thing it
// does: the work in its middle cost prompts 4 to 8 us of 40.  The questions cost
// them 1 us of 39 and 2 of 125; a step of 8 tokens and 504 padding rows behind
// them takes 4.2 us instead of 2.8, a step without padding no more than before.
// ---------------------------------------------------------------------------
constexpr int kReach = 256;

// The nearest token that is stored among `from`, from + step, ... (kReach of
// them); -1 if there is none.  Every lane of the warp calls it.
__device__ __noinline__ int nearest_stored(const RopeAppendParams& p, int from, int step) {
    constexpr int B = kReach / 32;
    const int lane = threadIdx.x & 31;
    const int64_t limit = static_cast<int64_t>(p.num_blocks) * p.block_size;
    int64_t slots[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {  // all loads on their way before any is used
        const int t = from + step * (32 * j + lane);
        slots[j] = t >= 0 && t < p.num_tokens ? p.slot_mapping[t] : -1;
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const int t = from + step * (32 * j + lane);
        const bool stored = slots[j] >= 0 && slots[j] < limit && !(p.positions && p.positions[t] < 0);
        const unsigned any = __ballot_sync(0xffffffffu, stored);
        if (any) return from + step * (32 * j + __ffs(any) - 1);
    }
    return -1;
}

// Whether the slot is one of the block's that starts at slot b: any (first = 0)
// or any but the first (1).
__device__ __forceinline__ bool in_block(const RopeAppendParams& p, int64_t slot, int64_t b, int first) {
    return slot >= b + first && slot < b + p.block_size;
}

// Whether the nearest token before t that is stored lies in the block at slot b.
__device__ __noinline__ bool block_before(const RopeAppendParams& p, int t, int64_t b) {
    bool unused = false;
    t = nearest_stored(p, t - 1, -1);
    return t >= 0 && in_block(p, slot_of(p, t, &unused), b, 0);
}

// The next run of the block at slot b at token t or after it: its first token,
// -1 if there is none.
__device__ __noinline__ int later_run(const RopeAppendParams& p, int t, int64_t b) {
    bool unused = false;
    t = t < p.num_tokens ? nearest_stored(p, t, 1) : -1;
    return t >= 0 && in_block(p, slot_of(p, t, &unused), b, 1) ? t : -1;
}

// Slot s0 at token t0 and the n - 1 tokens after it are a run that may go on: its
// length.  `open`: whether a later run of its block may follow, as far as the
// tokens read here tell.
__device__ __forceinline__ int run_length(const RopeAppendParams& p, int t0, int64_t s0, int off0, int n, bool& open) {
    const int lane = threadIdx.x & 31;
    while (true) {
        bool unused = false;
        const int64_t s = slot_of(p, t0 + n + lane, &unused);
        const bool in = n + lane < p.block_size - off0 && s == s0 + n + lane;
        const unsigned out = __ballot_sync(0xffffffffu, !in);
        const unsigned closed = __ballot_sync(0xffffffffu, t0 + n + lane >= p.num_tokens ||
                                                               (s >= 0 && !in_block(p, s, s0 - off0, 1)));
        const int k = out ? __ffs(out) - 1 : 32;
        n += k;
        if (out) {
            open = !(closed >> k & 1);
            return n;
        }
    }
}

// The runs of the block whose first run starts at token t0, one after the other:
// block `part` of `split` takes its share of the (head, K or V) items, a warp the
// same ones of every run, so that it finds the codes and scales of the run before.
template <int ACT, int PAIRS>
__device__ __noinline__ void split_runs(const RopeAppendParams& p, int t0, int part, int split) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lpr = p.head_dim / 8, rp = 32 / lpr;
    const int r = lane / lpr, c = lane - r * lpr;
    const bool idle = r >= rp;
    bool unused = false;
    int64_t s0 = slot_of(p, t0, &unused), blk;
    int off0;
    divmod_u(s0, p.block_size, blk, off0);
    const int64_t b = s0 - off0;
    while (true) {
        const int n = run_length(p, t0, s0, off0, 1, unused);
        for (int it = part * kWarps + warp; it < 2 * p.num_kv_heads; it += split * kWarps) {
            const bool is_k = it < p.num_kv_heads;
            const int head = is_k ? it : it - p.num_kv_heads;
            const int64_t tile = blk * p.num_kv_heads + head;
            RunRows run;
            run.stride = is_k ? p.k_stride : p.v_stride;
            run.src = static_cast<const uint16_t*>(is_k ? p.k : p.v) + t0 * run.stride + head * p.head_dim;
            run.scale = (is_k ? p.k_scales : p.v_scales) + tile;
            run.tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + tile * p.block_size * p.head_dim;
            run.positions = is_k && PAIRS != kPairsNone ? p.positions + t0 : nullptr;
            const float old = off0 == 0 ? 0.f : *run.scale;
            const float now = new_scale(run_top<ACT, PAIRS>(p, run, n, r, rp, c, idle), old);
            run_codes<ACT, PAIRS>(p, run, n, off0, r, rp, c, idle, now);
            __syncwarp();  // every lane has read the old scale
            if (now != old) {
                if (lane == 0) *run.scale = now;
                if (old > 0.f) requantise(run.tile, p.block_size, lpr, off0, n, __fdiv_rn(old, now), lane, 32);
            }
        }
        __syncwarp();  // before the next run's reads
        t0 = later_run(p, t0 + n, b);
        if (t0 < 0) return;
        s0 = slot_of(p, t0, &unused);
        off0 = static_cast<int>(s0 - b);
    }
}

template <int ACT, int PAIRS, int GROUP, int W>
__device__ __noinline__ void careful_block(const RopeAppendParams& p, int window, int w, int from, int part, int split,
                                           float* table);

// Runs that start in window w of `window` < 32 tokens: block `part` of `split`
// takes its share of each run's (head, K or V) items.  cos and sin of the run's
// tokens are computed once into shared memory.  CAREFUL: of the tokens from
// `from` on, where a block's tokens may be several runs.  GROUP == 1: windows of
// one token.
template <int ACT, int PAIRS, int GROUP, int W, bool CAREFUL = false>
__device__ __forceinline__ void scaled_block(const RopeAppendParams& p, int window, int w, int part, int split,
                                             float* table, int from = 0) {
    __shared__ float tops2[2 * kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lpr = p.head_dim / 8;
    const int lane_row = lane / lpr, chunk = lane - lane_row * lpr;
    // lane l holds token first - 1 + l: the window's tokens, the one before and some after
    const int first = w * window;
    bool bad = false;
    const int64_t slot = slot_of(p, first - 1 + lane, &bad);
    if (!CAREFUL && bad && lane >= 1 && lane <= window && warp == 0 && part == 0) atomicOr(p.err, kErrBadSlot);
    int64_t blk = 0;
    int off = 0;
    if (slot >= 0) divmod_u(slot, p.block_size, blk, off);
    // joined: the token continues the run of the one before it; close: it comes, inside a block, behind
    // a token of the block or a skipped one
    const int64_t prev = __shfl_up_sync(0xffffffffu, slot, 1);
    const int block = slot >= 0 ? static_cast<int>(blk) : -1, prev_block = __shfl_up_sync(0xffffffffu, block, 1);
    const unsigned joined = __ballot_sync(0xffffffffu, lane > 0 && slot >= 0 && prev == slot - 1 && off != 0);
    const unsigned close = __ballot_sync(
        0xffffffffu, off != 0 && first + lane > 1 && (prev_block == block || prev_block < 0));
    const unsigned starts = __ballot_sync(0xffffffffu, lane > 0 && slot >= 0) & ~joined;
    constexpr bool STEP = GROUP == 1;  // windows of one token
    if (!CAREFUL && !STEP && (close & starts))
        return careful_block<ACT, PAIRS, GROUP, W>(p, window, w, first, part, split, table);
    unsigned leaders = starts & (STEP ? 2u : (2u << window) - 2);
    if (CAREFUL) leaders &= ~0u << (from - first + 1);
    for (; leaders; leaders = STEP ? 0u : leaders & (leaders - 1)) {
        const int at = STEP ? 1 : __ffs(leaders) - 1;
        const int t0 = first - 1 + at;
        const int64_t s0 = __shfl_sync(0xffffffffu, slot, at), b0 = __shfl_sync(0xffffffffu, blk, at);
        const int off0 = __shfl_sync(0xffffffffu, off, at);
        if ((CAREFUL || STEP) && (close >> at & 1) && block_before(p, t0, s0 - off0)) continue;  // a later run
        // the run's length: the lanes joined after it, and further where it reaches the last lane
        const unsigned after = at < 31 ? ~(joined >> (at + 1)) : ~0u;
        int n = 1 + min(__ffs(after) - 1, 31 - at);
        bool open = !(starts >> at >> 1) && t0 + n < p.num_tokens;  // what starts next is not held
        if (at + n == 32) n = run_length(p, t0, s0, off0, n, open);
        if constexpr (CAREFUL) {
            if (later_run(p, t0 + n, s0 - off0) >= 0) {
                split_runs<ACT, PAIRS>(p, t0, part, split);
                continue;
            }
        } else if (STEP ? (open || (close & starts & ~3u)) && later_run(p, t0 + n, s0 - off0) >= 0 : open) {
            // (if not a step: the window's last leader)
            if constexpr (STEP) return split_runs<ACT, PAIRS>(p, t0, part, split);
            else return careful_block<ACT, PAIRS, GROUP, W>(p, window, w, t0, part, split, table);
        }
        if constexpr (PAIRS != kPairsNone) {
            // the rows that a run of GROUP passes has (at most kTable holds them)
            const Table<PAIRS> tab(p);
            __syncthreads();  // the run before is done with the table
            tab.fill(p, table, t0, min(n, GROUP * W * (32 / lpr)));
            __syncthreads();
        }
        const int items = 2 * p.num_kv_heads;
        if (GROUP == 1 && n == 1 && (lpr & (lpr - 1)) == 0) {
            const int rp = 32 / lpr;
            for (int it = (part * kWarps + warp) * rp; it < items; it += split * kWarps * rp)
                single_rows<ACT, PAIRS>(p, t0, b0, off0, it, table);
            continue;
        }
        constexpr int TEAMS = kWarps / W;
        int flip = 0;  // the pair's maxima alternate between two places
        for (int it = part * TEAMS + warp / W; it < items; it += split * TEAMS, flip ^= kWarps) {
            const bool is_k = it < p.num_kv_heads;
            const int head = is_k ? it : it - p.num_kv_heads;
            const int64_t tile = b0 * p.num_kv_heads + head;
            RunRows run;
            run.stride = is_k ? p.k_stride : p.v_stride;
            run.src = static_cast<const uint16_t*>(is_k ? p.k : p.v) + t0 * run.stride + head * p.head_dim;
            run.scale = (is_k ? p.k_scales : p.v_scales) + tile;
            run.tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + tile * p.block_size * p.head_dim;
            run.positions = is_k && PAIRS != kPairsNone ? p.positions + t0 : nullptr;
            if (PAIRS != kPairsNone && is_k)
                scaled_run<ACT, PAIRS, GROUP, W, PAIRS != kPairsNone>(p, run, n, off0, lane_row, chunk, table, tops2 + flip);
            else
                scaled_run<ACT, PAIRS, GROUP, W, false>(p, run, n, off0, lane_row, chunk, table, tops2 + flip);
        }
        if (W == 2) __syncthreads();  // the places of the last maxima
    }
}

template <int ACT, int PAIRS, int GROUP, int W>
__device__ __noinline__ void careful_block(const RopeAppendParams& p, int window, int w, int from, int part, int split,
                                           float* table) {
    scaled_block<ACT, PAIRS, GROUP, W, true>(p, window, w, part, split, table, from);
}

// Items (token, part of its rows) of block `cta`, one a warp: at most kWarps tokens.
template <int ACT, int CACHE, int PAIRS>
__device__ __forceinline__ void rows_block(const RopeAppendParams& p, int cta, int parts, int per, int rows, float* table) {
    const int warp = threadIdx.x >> 5;
    const int64_t item0 = static_cast<int64_t>(cta) * kWarps;
    int64_t token0, token, last;
    int unused, part;
    divmod_u(item0, parts, token0, unused);
    divmod_u(item0 + warp, parts, token, part);
    divmod_u(item0 + kWarps - 1, parts, last, unused);
    const int tokens = static_cast<int>(min(last, static_cast<int64_t>(p.num_tokens) - 1) - token0) + 1;
    Table<PAIRS>(p).fill(p, table, token0, tokens);
    __syncthreads();
    if (token >= p.num_tokens || p.positions[token] < 0) return;  // padding: q_out keeps its row
    plain_rows<ACT, CACHE, PAIRS>(p, static_cast<int>(token), part * per, min(rows, part * per + per),
                                  table, static_cast<int>(token - token0));
}

// How a launch divides its work.
struct Split {
    int window, windows, share;  // runs: tokens a window, windows, blocks a window
    int parts, per, rows;        // rows: items a token, rows an item, rows a token
};

template <int ACT, int CACHE, int PAIRS>
__global__ void __launch_bounds__(kWarps * 32, 3) rope_rows_kernel(const RopeAppendParams p, const Split d) {
    __shared__ __align__(16) float table[kTable];
    rows_block<ACT, CACHE, PAIRS>(p, blockIdx.x, d.parts, d.per, d.rows, table);
    // launched beside the kernel that stores the keys and values: done when that is done
    if (CACHE == kE4M3B) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Prompts: runs of many tokens.  What bounds it is instructions (56 % of the
// issue slots, a quarter of the memory's rate; 44 us for 17,700 tokens of 2 x 8
// heads, rotated).  The queries' rows follow in a launch of their own that
// starts as these blocks drain (88 us, 6.6 TB/s): one grid that mixes both kinds
// of blocks took 130 us instead of 125, the rows having fewer blocks a SM there.
template <int ACT, int PAIRS>
__global__ void __launch_bounds__(kWarps * 32, PAIRS == kPairsNone ? 4 : 3) scaled_runs_kernel(const RopeAppendParams p, const Split d) {
    __shared__ __align__(16) float table[PAIRS == kPairsNone ? 4 : kTable];
    asm volatile("griddepcontrol.launch_dependents;");
    const int w = blockIdx.x / d.share;
    scaled_block<ACT, PAIRS, PAIRS == kPairsNone ? 8 : 4, 2>(p, d.window, w, blockIdx.x - w * d.share, d.share, table);
}

// Few tokens (a decode step): runs and rows in one launch.  What bounds it is
// its round trips to memory, one after the other: the slots, then the old scale
// and the row, and for a block whose scale grows its codes (256 tokens of 2 x 40
// heads 7.4 us, 1.2 us of them bytes; 12.9 us with a warp for each row and the
// codes loaded one piece at a time).
template <int ACT, int PAIRS>
__global__ void __launch_bounds__(kWarps * 32, 3) scaled_step_kernel(const RopeAppendParams p, const Split d) {
    __shared__ __align__(16) float table[PAIRS == kPairsNone ? 4 : kTable];
    const int cta = blockIdx.x, runs = d.windows * d.share;
    if (cta < runs) {
        const int w = cta / d.share;
        scaled_block<ACT, PAIRS, 1, 1>(p, d.window, w, cta - w * d.share, d.share, table);
    } else {
        if constexpr (PAIRS != kPairsNone) rows_block<ACT, kE4M3B, PAIRS>(p, cta - runs, d.parts, d.per, d.rows, table);
    }
}

template <int ACT, int CACHE, int PAIRS>
cudaError_t launch(const RopeAppendParams& p, cudaStream_t stream) {
    static_assert(kWarps * 2 * 8 * 32 <= kTable, "a block's tokens fit the table at rotary_dim 256");
    const int rp = 32 / (p.head_dim / 8);
    Split d{};
    d.rows = p.positions == nullptr ? 0 : CACHE == kE4M3B ? p.num_q_heads : p.num_q_heads + 2 * p.num_kv_heads;
    // rows of a token per warp: all of them when the tokens alone fill the GPU
    const int passes = (d.rows + rp - 1) / rp;
    int split = 1;
    while (split < passes && static_cast<int64_t>(p.num_tokens) * split < kFill * kWarps) split *= 2;
    d.per = d.rows ? (passes + split - 1) / split * rp : 1;
    d.parts = d.rows ? (d.rows + d.per - 1) / d.per : 1;
    const int64_t row_blocks = d.rows ? (static_cast<int64_t>(p.num_tokens) * d.parts + kWarps - 1) / kWarps : 0;
    if (row_blocks > 0x3fffffff) return cudaErrorInvalidConfiguration;
    const unsigned threads = kWarps * 32;
    if constexpr (CACHE != kE4M3B) {
        rope_rows_kernel<ACT, CACHE, PAIRS><<<static_cast<unsigned>(row_blocks), threads, 0, stream>>>(p, d);
        return cudaGetLastError();
    } else {
        // prompts: a window starts a run or a few, whose heads one block works off; few tokens: one token a window
        d.window = 16;
        while (d.window > 1 && (p.num_tokens + d.window - 1) / d.window < kFill) d.window /= 2;
        d.windows = (p.num_tokens + d.window - 1) / d.window;
        const int per_block = d.window == 1 && (rp & (rp - 1)) == 0 ? kWarps * rp : kWarps;
        const int most = (2 * p.num_kv_heads + per_block - 1) / per_block;
        d.share = 1;
        const int fill = d.window == 1 ? 4 * kFill : kFill;
        while (d.share < most && static_cast<int64_t>(d.windows) * d.share < fill) ++d.share;
        const int64_t run_blocks = static_cast<int64_t>(d.windows) * d.share;
        if (run_blocks + row_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
        if (d.window == 1) {
            scaled_step_kernel<ACT, PAIRS><<<static_cast<unsigned>(run_blocks + row_blocks), threads, 0, stream>>>(p, d);
            return cudaGetLastError();
        }
        scaled_runs_kernel<ACT, PAIRS><<<static_cast<unsigned>(run_blocks), threads, 0, stream>>>(p, d);
        cudaError_t e = cudaGetLastError();
        if constexpr (PAIRS != kPairsNone) {
            if (e != cudaSuccess || row_blocks == 0) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(row_blocks));
            cfg.blockDim = dim3(threads);
            cfg.stream = stream;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, rope_rows_kernel<ACT, CACHE, PAIRS>, p, d);
        }
        return e;
    }
}

template <int ACT, int CACHE>
cudaError_t by_pairs(const RopeAppendParams& p, cudaStream_t s) {
    if (p.positions == nullptr) {
        if constexpr (CACHE == kE4M3B) return launch<ACT, CACHE, kPairsNone>(p, s);
        else return cudaErrorInvalidValue;
    }
    if (p.interleaved) return launch<ACT, CACHE, kPairsNext>(p, s);
    return p.rotary_dim % 16 == 0 ? launch<ACT, CACHE, kPairsChunks>(p, s) : launch<ACT, CACHE, kPairsApart>(p, s);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int act, int cache, cudaStream_t s) {
    if (act == kF16)
        return cache == kF16     ? by_pairs<kF16, kF16>(p, s)
               : cache == kE4M3  ? by_pairs<kF16, kE4M3>(p, s)
               : cache == kE4M3B ? by_pairs<kF16, kE4M3B>(p, s)
                                 : cudaErrorInvalidValue;
    return cache == kBF16    ? by_pairs<kBF16, kBF16>(p, s)
           : cache == kE4M3  ? by_pairs<kBF16, kE4M3>(p, s)
           : cache == kE4M3B ? by_pairs<kBF16, kE4M3B>(p, s)
                             : cudaErrorInvalidValue;
}

}  // namespace pkv
