// kv_attn.hip -- causal attention over the paged 4-bit cache.
//
//   out = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q.k_t),
// over the visible tokens, in one pass with a running maximum.
//
// Both products run on the 16x16x32 fp16 MFMA with the cached tokens' codes
// turned into fp16 levels on the way in, and with the scales kept out of it:
//   S^T = K Q^T   A = the levels of 16 tokens, B = 16 query rows; the sum of
//                 each 64-element block is scaled by the block's absmax in fp32;
//   O^T = V^T P^T A = the levels of 16 elements over 32 tokens, B = the
//                 softmax weights times the block's absmax.
// The result of the first product is already laid out as the second one's B
// operand (lane: query l%16, tokens 4(l/16) .. +3 of each half tile), so the
// weights never leave their registers.
//
// Levels, not products: fp16 holds the levels eight times better than bf16
// would hold scale * level, and one table then serves every block.  It lies in
// LDS once per lane ([256 code bytes][64 lanes] of two levels each): a lookup
// turns one byte of codes into one packed operand register with one byte
// permute for the address and one conflict-free read.  Keys are looked up as
// they lie (two elements of a token); for values the nibbles of two tokens are
// exchanged first, so that a byte holds one element of both.
//
// Weights: fp16 has to hold p_t * absmax_t, whatever the size of the cached
// values.  The running maximum M is therefore taken over z_t = log2 p_t + the
// exponent of the largest absmax of the token's blocks: 2^(log2 p_t - M) *
// absmax_t is then at most 1, and the sum of the softmax keeps the same factor
// in fp32.  M is moved only when a tile exceeds it by more than 6, and 2^8
// more puts the weights in the upper part of fp16's range: the largest is between
// 2^7 and 2^14, so that all down to 2^-21 of it have fp16's full precision.
//
// Work: a unit is a block of query rows of one request and cache head.  Rows
// are (query, head of the group) pairs, so the heads that share a cache head
// share its reads.  With few rows the waves of a workgroup take turns at the
// tokens and join at the end (k_attn_few), or, if there are units for every wave,
// each has its own (k_attn_alone); with many rows each wave has some of a unit's
// (k_attn_many).
#include <algorithm>

#include "kv_device.h"

using namespace nf4dev;

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;             // tokens of one step
constexpr float kLazy = 6.0f;         // how far a tile may exceed the running maximum (log2)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kBias = 8.0f;         // log2 of the largest weight when the maximum was last moved
constexpr float kLeast = 0x1p-90f;    // a smaller absmax has this one's exponent

__device__ __forceinline__ f32x4_t mfma_f16(const u32x4_t& a, const u32x4_t& b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    f16x2_t p;
    p[0] = (_Float16)a;
    p[1] = (_Float16)b;
    return __builtin_bit_cast(uint32_t, p);
}

// a * b, and 0 where either is 0, whatever the other: v_mul_legacy_f32.  (The
// intrinsic, since the compiler keeps the wait that a result of v_exp_f32
// needs before its use only for instructions that it issues itself.)
extern "C" __device__ __attribute__((const)) float kv_mul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float mul_zero(float a, float b) { return kv_mul_legacy(a, b); }

__device__ __forceinline__ float exp2f_(float x) { return __builtin_amdgcn_exp2f(x); }

// The table holds the levels times a constant whose inverse goes into the
// fp32 sums.  FP4 levels times 6 are fp16 numbers.  For NF4 the constant was
// searched (2^24 values in [1, 2)) for one that brings all sixteen close to
// fp16 numbers: they are off by at most 6.2e-5 of the absmax instead of
// 1.9e-4, and by 1.7e-6 instead of 1.1e-5 in the mean over the codes of normal
// data.  The mean is what a sum over 10^5 tokens keeps: with a constant of 1
// the result of such a sum was off by 4.6e-3, its bf16 rounding by 1.7e-3.
constexpr float kNf4Times = 1.4589563608169556f;
__host__ __device__ constexpr float level_unit(int qt) { return qt ? 1.0f / 6.0f : 1.0f / kNf4Times; }
inline uint32_t level_f16(int qt, int i) {
    const float v = __builtin_bit_cast(float, qt_level_bits(qt, i));
    return __builtin_bit_cast(uint16_t, (_Float16)(qt ? rintf(12.0f * v) * 0.5f : v * kNf4Times));
}

struct Params {
    const uint8_t* codes[2];
    const uint16_t* scales[2];
    uint32_t n_pages;
    int n_heads, pshift, qt;
    uint32_t levels[8];  // level_f16 of codes 2i and 2i + 1
    kv::Attn a;
    int group;       // query heads per cache head
    int row_blocks;  // blocks of query rows of a request
    kv::Div by_group, by_row_blocks, by_heads, by_splits;
    int shares;      // few rows: workgroups per head that share the tiles evenly; 0: one per (request, block)
    int step;        // few rows: a workgroup's next unit
    int splits;      // many rows: workgroups that share the tiles of a (request, block)
    float* part;     // partial results: [share][head][2][NT][part_floats(D)], or [block][split][head][8 NT][part_floats(D)]
    int zero_rest;   // rows that are not computed get zeros
    int4* cuts;      // [share][head]: the unit that goes on in later shares: the last one, q0, rows, row0
};

// The tiles a block of query rows visits: the tiles of the first tokens that
// stay visible, then those from the window's start to the last position.
struct Tiles {
    int first_end;       // tiles [0, first_end)
    int start, end;      // tiles [start, end)
    __device__ int count() const { return first_end + end - start; }
    __device__ int at(int i) const { return i < first_end ? i : start + i - first_end; }
};

// p0, p1: positions of the block's first and last query; T: tokens of a tile
template <int T = kTile>
__device__ __forceinline__ Tiles tiles_of(int p0, int p1, int window, int sinks) {
    Tiles t = {0, 0, 0};
    if (p1 < 0) return t;
    t.end = p1 / T + 1;
    if (window > 0) {
        const int64_t lo = int64_t(p0) - window + 1;
        t.start = lo > 0 ? int(lo / T) : 0;
        const int seen = sinks < p1 + 1 ? sinks : p1 + 1;
        const int fe = (seen + T - 1) / T;
        t.first_end = fe < t.start ? fe : t.start;
    }
    return t;
}

// A block of query rows of one request: what a workgroup works on at a time.
struct Unit {
    int request, q0;   // its first query's row of q
    int rows, row0;    // rows of the request; the block's first
    int first_pos;     // position of query 0 (negative: it sees nothing)
    Tiles tiles;
    bool empty;        // no such rows
};

// What a request's unit is made from: its queries and its length.
struct Lengths { int c0, c1, have; };

// UNIFORM: the request is the same for the wave (the lengths are then scalars).
template <bool UNIFORM>
__device__ __forceinline__ Lengths lengths_of(const Params& p, int request) {
    if constexpr (UNIFORM) {
        typedef const __attribute__((address_space(4))) int32_t constant_t;
        constant_t* cu = (constant_t*)(uintptr_t)p.a.cu_q;
        constant_t* lens = (constant_t*)(uintptr_t)p.a.kv_lens;
        return {cu[request], cu[request + 1], lens[request]};
    }
    return {p.a.cu_q[request], p.a.cu_q[request + 1], p.a.kv_lens[request]};
}

template <int T = kTile>
__device__ __forceinline__ Unit unit_of(const Params& p, int u, int block_rows, int request, const Lengths& a) {
    Unit x;
    x.request = request;
    // the longest blocks of a request come first
    const int block = p.row_blocks - 1 - (u - request * p.row_blocks);
    const int total = int(p.a.total_q);
    const int lo = min(max(a.c0, 0), total), hi = min(max(a.c1, lo), total);
    const int n = hi - lo, len = min(max(a.have, 0), p.a.max_len);
    x.q0 = lo;
    x.rows = min(n, p.a.max_q) * p.group;
    x.row0 = block * block_rows;
    x.first_pos = len - n;  // (a query past max_q is not computed, but the last query is the last token)
    x.empty = x.row0 >= x.rows;
    x.tiles = Tiles{0, 0, 0};
    if (!x.empty)
        x.tiles = tiles_of<T>(x.first_pos + p.by_group.of(x.row0),
                           x.first_pos + p.by_group.of(min(x.row0 + block_rows, x.rows) - 1), p.a.window, p.a.sinks);
    return x;
}

template <bool UNIFORM, int T = kTile>
__device__ __forceinline__ Unit unit_of(const Params& p, int u, int block_rows) {
    const int request = p.by_row_blocks.of(u);
    return unit_of<T>(p, u, block_rows, request, lengths_of<UNIFORM>(p, request));
}

// ---------------------------------------------------------------------------
// One wave's part: NT tiles of 16 query rows against a list of token tiles.
template <int D, int NT>
struct Wave {
    static constexpr int NB = D / 64;            // blocks of an entry

    const Params& p;
    const char* table;  // in LDS: entry e, copy of lane i, at e * 256 + i * 4
    const u32x4_t (*qs)[NB][2][64];  // in LDS: the operands of the queries at hand
    int head, l, c, g;  // lane; query (or token, or element) of a fragment; k group
    int key_at, value_at, scale_at;  // the lane's offsets in a half tile
    float f[NT];        // what a sum of products is worth in log2 units
    int pos[NT];        // position of this lane's row
    int pos_first, pos_last;  // of the wave's rows
    f32x4_t o[NT][NB][4];     // O^T: element 64n + 16g + 4r + i of query c in o[t][n][i][r]
    float M[NT], sum[NT];

    // one tile's codes and scales, as loaded
    struct Keys {
        u32x2_t k[2][NB];        // token 16h + c, elements 64n + 16g .. +15
        uint32_t s[2][2 * NB];   // absmax of tokens 16h + 4g .. +3, NB each (bf16)
    };
    struct Values {
        uint32_t v[8][NB];       // token 16h + 4g + j at 4h + j: elements 64n + 4c .. +3 (16 bits)
        uint32_t s[2][2 * NB];
    };

    __device__ __forceinline__ Wave(const Params& p_, const char* table_, const u32x4_t (*qs_)[NB][2][64], int head_)
        : p(p_), table(table_), qs(qs_), head(head_) {
        l = threadIdx.x & 63;
        c = l & 15;
        g = l >> 4;
        key_at = c * (D / 2) + 8 * g;
        value_at = 4 * g * (D / 2) + 2 * c;
        scale_at = 8 * g * NB;
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            M[t] = -INFINITY;
            sum[t] = 0.0f;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][n][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }

    // A row of queries: loaded as it lies, then written to `dst` as an fp16
    // operand scaled by a power of two, whose factor is returned.
    struct Row { u32x4_t raw[NB][2]; };
    static __device__ __forceinline__ void load_row(const Params& p, const Unit& x, int row, int head, Row& q) {
        const int g = (threadIdx.x >> 4) & 3;
        const int r = min(row, x.rows - 1), qi = p.by_group.of(r);
        const uint16_t* at = p.a.q + int64_t(x.q0 + qi) * p.a.q_stride + int64_t(head * p.group + (r - qi * p.group)) * D;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int s = 0; s < 2; ++s) q.raw[n][s] = *reinterpret_cast<const u32x4_t*>(at + 64 * n + 16 * g + 8 * s);
    }
    template <typename Put>
    static __device__ __forceinline__ float stage_row(const Params& p, const Row& q, Put put) {
        uint32_t mb = 0;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mb = max(mb, max(q.raw[n][s][i] & 0x7fffu, (q.raw[n][s][i] >> 16) & 0x7fffu));
        mb = max(mb, uint32_t(__shfl_xor(int(mb), 16, 64)));
        mb = max(mb, uint32_t(__shfl_xor(int(mb), 32, 64)));
        const int e = max(int(mb >> 7), 1) - 127;  // exponent of the row's largest
        const float f = ldexpf(p.a.scale * kLog2e * level_unit(p.qt), e);
        // a row holding Inf or NaN is NaN throughout, and one whose factor
        // vanishes is 0 (so that f * -inf is -inf in every row)
        const bool bad = mb >= 0x7f80u, none = f == 0.0f;
        const uint32_t fill = bad ? 0x7e007e00u : 0u;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4_t v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = pack_f16(ldexpf(bf16_lo(q.raw[n][s][i]), -e), ldexpf(bf16_hi(q.raw[n][s][i]), -e));
                    v[i] = bad || none ? fill : v[i];
                }
                put(n, s, v);
            }
        return bad || none ? 1.0f : f;
    }

    __device__ __forceinline__ void place(const Unit& x, int row0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) pos[t] = x.first_pos + p.by_group.of(min(row0 + 16 * t + c, x.rows - 1));
        pos_first = x.first_pos + p.by_group.of(row0);
        pos_last = x.first_pos + p.by_group.of(min(row0 + 16 * NT, x.rows) - 1);
    }

    __device__ __forceinline__ uint32_t look(uint32_t word, int byte) const {
        const uint32_t at = __builtin_amdgcn_perm(word, uint32_t(l) * 4u, 0x0C0C0000u | (uint32_t(4 + byte) << 8));
        return *reinterpret_cast<const uint32_t*>(table + at);
    }

    // absmax of block n of token r of the lane's four
    static __device__ __forceinline__ float scale_of(const uint32_t (&s)[2 * NB], int r, int n) {
        const int i = r * NB + n;
        return (i & 1) ? bf16_hi(s[i >> 1]) : bf16_lo(s[i >> 1]);
    }

    // first entry of half h of a tile, given its page
    __device__ __forceinline__ int64_t entry(uint32_t page, int t0) const {
        return ((int64_t(page < p.n_pages ? page : 0u) * p.n_heads + head) << p.pshift) + (t0 & ((1 << p.pshift) - 1));
    }

    // Buffer loads: the half tile's address in scalar registers, one offset
    // register a lane, and the rest in the instruction.  With live == 0 the
    // buffer is empty and nothing is read, so that a walk's last step needs no
    // branch around its loads.  (Each offset passes through an empty asm, or
    // its sums with constants would be made ahead, one register for each.)
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* at, uint32_t bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(at), 0, int(bytes), 0x00020000);
    }

    __device__ __forceinline__ void load_scales(const uint16_t* base, uint32_t live, uint32_t (&s)[2 * NB]) {
        const auto r = buffer(base, live * (16 * NB * 2));
        asm volatile("" : "+v"(scale_at));
        if constexpr (NB == 1) {
            const u32x2_t a = __builtin_amdgcn_raw_buffer_load_b64(r, scale_at, 0, 0);
            s[0] = a[0], s[1] = a[1];
        } else {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) {
                const u32x4_t a = __builtin_amdgcn_raw_buffer_load_b128(r, scale_at + 16 * i, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) s[4 * i + k] = a[k];
            }
        }
    }

    __device__ __forceinline__ void load_keys(int tile, const uint32_t (&page)[2], uint32_t live, Keys& r) {
        asm volatile("" : "+v"(key_at));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = entry(page[h], tile * kTile + 16 * h);
            const auto kc = buffer(p.codes[0] + at * (D / 2), live * (16 * (D / 2)));
#pragma unroll
            for (int n = 0; n < NB; ++n)
                r.k[h][n] = __builtin_amdgcn_raw_buffer_load_b64(kc, key_at + 32 * n, 0, 0);
            load_scales(p.scales[0] + at * NB, live, r.s[h]);
        }
    }

    __device__ __forceinline__ void load_values(int tile, const uint32_t (&page)[2], uint32_t live, Values& r) {
        asm volatile("" : "+v"(value_at));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = entry(page[h], tile * kTile + 16 * h);
            const auto vc = buffer(p.codes[1] + at * (D / 2), live * (16 * (D / 2)));
            load_scales(p.scales[1] + at * NB, live, r.s[h]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    r.v[4 * h + j][n] = __builtin_amdgcn_raw_buffer_load_b16(vc, value_at + j * (D / 2) + 32 * n, 0, 0);
        }
    }

    // S^T by half tile: products of tokens 16h + 4g + r over each block of
    // elements, in two steps.  a[n]: the operands of step s; query(t, n): of the queries
    typedef f32x4_t Products[NT][NB];
    template <typename Q>
    static __device__ __forceinline__ void multiply(const u32x4_t (&a)[NB], Q query, int s, Products& acc) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                acc[t][n] = mfma_f16(a[n], query(t, n), s ? acc[t][n] : f32x4_t{0.f, 0.f, 0.f, 0.f});
    }
    // Their sums, scale(r, n) being the absmax: times f they are scores in log2 units.
    template <typename S>
    static __device__ __forceinline__ void add_up(const Products& acc, S scale, int h, float (&s2)[NT][2][4]) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = scale(r, 0) * acc[t][0][r];
#pragma unroll
                for (int n = 1; n < NB; ++n) v = __builtin_fmaf(scale(r, n), acc[t][n][r], v);
                s2[t][h][r] = v;
            }
    }

    __device__ __forceinline__ u32x4_t look_up(uint32_t word) const {
        return u32x4_t{look(word, 0), look(word, 1), look(word, 2), look(word, 3)};
    }

    // Every row of the wave sees every token of the tile.
    // there: whether the pages of its halves exist
    __device__ __forceinline__ bool whole(int tile, const bool (&there)[2]) const {
        const int t0 = tile * kTile;
        return there[0] && there[1] && t0 + kTile - 1 <= pos_first &&
               (p.a.window == 0 || t0 > before_window(pos_last) || t0 + kTile <= p.a.sinks);
    }

    // The last token before the window of a row at position q; for a row that
    // stands before the first token, and sees nothing anyway, that of the first
    // (its own would not fit 31 bits with the largest windows).
    __device__ __forceinline__ int before_window(int q) const { return max(q, 0) - p.a.window; }

    // A score that becomes -inf for the tokens that a row does not see.
    __device__ __forceinline__ void hide(int tile, const bool (&there)[2], float (&s2)[NT][2][4]) const {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float hidden = f[t] < 0.0f ? INFINITY : -INFINITY;
            const int after = p.a.window ? before_window(pos[t]) : -1;  // tokens up to this one are hidden
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = tile * kTile + 16 * h + 4 * g + r;
                    const bool in = there[h] & (tok <= pos[t]) & ((tok > after) | (tok < p.a.sinks));
                    s2[t][h][r] = in ? s2[t][h][r] : hidden;
                }
        }
    }

    // exponent of the largest absmax of a token's blocks (a NaN one, which makes
    // its block's outputs NaN by itself, is passed over)
    static __device__ __forceinline__ float exponent_of(float m) {
        return float(__builtin_amdgcn_frexp_expf(fmaxf(m, kLeast)));
    }

    // The running softmax moves on by one tile, whose weights times absmax
    // become operands.  scale(h, r, n): the absmax; e(h, r): their exponent
    template <typename S, typename E>
    __device__ __forceinline__ void weigh(S scale, E e, const float (&s2)[NT][2][4], u32x4_t (&wt)[NT][NB]) {
        // (each lane looks at its own tokens; the rows' maxima are made only
        // when one of them has to move)
        float top[NT];
        bool moves = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            top[t] = __builtin_fmaf(s2[t][0][0], f[t], e(0, 0));
#pragma unroll
            for (int i = 1; i < 8; ++i)
                top[t] = fmaxf(top[t], __builtin_fmaf(s2[t][i >> 2][i & 3], f[t], e(i >> 2, i & 3)));
            moves |= top[t] > M[t] + kLazy;
        }
        if (__any(moves)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                top[t] = fmaxf(top[t], __shfl_xor(top[t], 16, 64));
                top[t] = fmaxf(top[t], __shfl_xor(top[t], 32, 64));
                // (a bound of the exact maximum, whatever the size of the scores)
                const float next = top[t] > M[t] + kLazy ? __builtin_fmaf(fabsf(top[t]), 0x1p-22f, top[t]) : M[t];
                const float by = next == -INFINITY ? 1.0f : exp2f_(M[t] - next);
                M[t] = next;
                sum[t] *= by;
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][n][i] *= by;
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float m = M[t] == -INFINITY ? 0.0f : M[t] - kBias;
            float wgt[NB][2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float pr = exp2f_(__builtin_fmaf(s2[t][h][r], f[t], -m));
                    sum[t] += pr;
                    // (a hidden token's absmax may be anything: 0 times it is 0 here)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        wgt[n][h][r] = mul_zero(pr, scale(h, r, n));
                }
#pragma unroll
            for (int n = 0; n < NB; ++n)
                wt[t][n] = u32x4_t{pack_f16(wgt[n][0][0], wgt[n][0][1]), pack_f16(wgt[n][0][2], wgt[n][0][3]),
                                   pack_f16(wgt[n][1][0], wgt[n][1][1]), pack_f16(wgt[n][1][2], wgt[n][1][3])};
        }
    }

    // The operands of block n of the values: element 4c + i of the tile's tokens
    // from the lane's bytes of eight of them.  put(i, operand)
    template <typename Put>
    __device__ __forceinline__ void turn_values(const uint32_t (&v)[8], Put put) const {
        // byte k of `even` (`odd`): elements 4c + 2k (+ 1) of two tokens, two
        // pairs of tokens to a word
        constexpr uint32_t HI = 0xf0f0f0f0u, LO = 0x0f0f0f0fu;
        uint32_t even[2], odd[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // tokens (0, 1) in the low half, (2, 3) in the high half
            const uint32_t a = v[4 * h] | (v[4 * h + 2] << 16);
            const uint32_t d = v[4 * h + 1] | (v[4 * h + 3] << 16);
            even[h] = (a & HI) | ((d >> 4) & LO);
            odd[h] = ((a << 4) & HI) | (d & LO);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t(&src)[2] = (i & 1) ? odd : even;
            put(i, u32x4_t{look(src[0], i >> 1), look(src[0], 2 + (i >> 1)), look(src[1], i >> 1),
                           look(src[1], 2 + (i >> 1))});
        }
    }

    // ---- a walk over the tiles list[first], list[first + step], ... below
    // list[last]: read_ids(), then begin(), which issues the first tile's
    // loads (either may come long before the next), then run().  Keys are loaded
    // again as soon as they are used up, and so are values: each load has the
    // other half of a step to arrive.
    Keys keys;
    Values values;
    uint32_t ids[2];   // lane y: the pages of the walk's tile number 64k + y,
    uint32_t page[2];  // read 64 tiles at a time; the current tile's
    int tile;

    __device__ __forceinline__ void read_ids(const Unit& x, int i, int last, int step, uint32_t (&ids)[2]) const {
        if (i >= last) return;
        const int32_t* row = p.a.table + int64_t(x.request) * p.a.width;
        const int t = x.tiles.at(min(i + l * step, last - 1));
#pragma unroll
        for (int h = 0; h < 2; ++h)
            ids[h] = uint32_t(row[min((t * kTile + 16 * h) >> p.pshift, max(p.a.width - 1, 0))]);
    }

    __device__ __forceinline__ void begin(const Unit& x, int first, int last) {
        if (first >= last) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) page[h] = uint32_t(__builtin_amdgcn_readfirstlane(int(ids[h])));
        tile = __builtin_amdgcn_readfirstlane(x.tiles.at(first));
        load_keys(tile, page, 1, keys);
        load_values(tile, page, 1, values);
    }

    __device__ __forceinline__ void run(const Unit& x, int first, int last, int step) {
        for (int i = first, n = 1; i < last; i += step, ++n) {
            const bool more = i + step < last;
            if (more && (n & 63) == 0) read_ids(x, i + step, last, step, ids);
            uint32_t next[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) next[h] = uint32_t(__builtin_amdgcn_readlane(int(ids[h]), n & 63));
            const int then = more ? __builtin_amdgcn_readfirstlane(x.tiles.at(i + step)) : 0;
            // (read from LDS in every step: kept in registers they would cost a
            // wave of occupancy)
            int lane = l;
            asm volatile("" : "+v"(lane));
            float s2[NT][2][4];
            // (The lookups of both halves are under way together: 3 % of a call's
            // time at 128 elements a head.  At 256, where the registers do not hold
            // them, a block's at a time: all of them would be 5 to 20 % slower.)
            constexpr int kTogether = NB <= 2 ? 2 : 1;
#pragma unroll
            for (int h0 = 0; h0 < 2; h0 += kTogether) {
                u32x4_t a[kTogether][2][NB];
                if constexpr (kTogether == 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int n = 0; n < NB; ++n) a[h][s][n] = look_up(keys.k[h][n][s]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int h = h0; h < h0 + kTogether; ++h) {
                    Products acc;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if constexpr (kTogether == 1) {
#pragma unroll
                            for (int n = 0; n < NB; ++n) a[0][s][n] = look_up(keys.k[h][n][s]);
                        }
                        multiply(a[h - h0][s], [&](int t, int n) { return qs[t][n][s][lane]; }, s, acc);
                    }
                    add_up(acc, [&](int r, int n) { return scale_of(keys.s[h], r, n); }, h, s2);
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // (the keys' registers are free from here on)
            load_keys(then, next, more, keys);
            const bool there[2] = {page[0] < p.n_pages, page[1] < p.n_pages};
            if (!whole(tile, there)) hide(tile, there, s2);
            float e[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float m = scale_of(values.s[h], r, 0);
#pragma unroll
                    for (int n = 1; n < NB; ++n) m = fmaxf(m, scale_of(values.s[h], r, n));
                    e[h][r] = exponent_of(m);
                }
            u32x4_t wt[NT][NB];
            weigh([&](int h, int r, int n) { return scale_of(values.s[h], r, n); },
                  [&](int h, int r) { return e[h][r]; }, s2, wt);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                uint32_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = values.v[j][n];
                u32x4_t ready[4];  // (the sixteen lookups are under way together)
                turn_values(v, [&](int i, const u32x4_t& a) { ready[i] = a; });
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t) o[t][n][i] = mfma_f16(ready[i], wt[t][n], o[t][n][i]);
            }
            __builtin_amdgcn_sched_barrier(0);
            load_values(then, next, more, values);
            tile = then;
            page[0] = next[0], page[1] = next[1];
        }
    }

    __device__ __forceinline__ void close() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sum[t] += __shfl_xor(sum[t], 16, 64);
            sum[t] += __shfl_xor(sum[t], 32, 64);
        }
    }

    __device__ __forceinline__ void write(const Unit& x, int row0, int t) const {
        const int row = row0 + 16 * t + c;
        if (row >= x.rows) return;
        const float by = sum[t] == 0.0f ? 0.0f : level_unit(p.qt) / sum[t];
        const int qi = p.by_group.of(row);
        uint16_t* dst = p.a.out + int64_t(x.q0 + qi) * p.a.out_stride + int64_t(head * p.group + (row - qi * p.group)) * D;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float v[16];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * r + i] = o[t][n][i][r] * by;
            kv::store_bf16<16>(dst + 64 * n + 16 * g, v);
        }
    }
};

// ---- results of the same rows added up
// A result of 16 rows is D/16 quads of registers for each of 64 lanes, and {M,
// sum} of each row.  Quad 4n + i of lane (c, g) holds elements 64n + 16g + i +
// {0, 4, 8, 12} of row c.

// Stores a quad of a row's output, or does nothing past the unit's last row.
template <int D>
__device__ __forceinline__ void store_quad(const Params& p, int q0, int rows, int head, int row, int quad, int g,
                                           f32x4_t v, float total) {
    if (row >= rows) return;
    const float by = total == 0.0f ? 0.0f : level_unit(p.qt) / total;
    const int qi = p.by_group.of(row);
    uint16_t* dst = p.a.out + int64_t(q0 + qi) * p.a.out_stride + int64_t(head * p.group + (row - qi * p.group)) * D +
                    64 * (quad >> 2) + 16 * g + (quad & 3);
#pragma unroll
    for (int r = 0; r < 4; ++r) dst[4 * r] = to_bf16(v[r] * by);
}

// The waves of a workgroup add up their results of one tile of rows: each
// writes its quads to LDS, and each thread then adds one quad over the waves.
// Only the lanes of rows that exist take part, so that with 8 rows or fewer
// all quads of 128 elements fit at once.
template <int D, int NT, int NW>
struct Join {
    using W = Wave<D, NT>;
    static constexpr int kQuads = D / 16;
    // quads of 64 lanes a wave has room for (at D == 64 two workgroups share a CU's LDS)
    static constexpr int kPart = D == 256 ? 8 : D == 128 ? 4 : NT == 2 ? 4 : 1;
    struct Lds {
        f32x4_t quad[kPart * 64 * NW];
        float stat[2][NW][16];  // M, sum
    };

    // out(quad, lane, value, M, total) is called once for each quad and lane
    template <typename Out>
    static __device__ __forceinline__ void run(const W& wave, int t, int rows, int w, Lds& lds, Out out) {
        const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
        const int lanes = 4 * rows;  // of a quad
        // the thread's quad and lane (quotients below 2^10: the reciprocal's
        // error is far below the half that is added)
        const int item = int(threadIdx.x);
        const float inv = __builtin_amdgcn_rcpf(float(rows));
        const int at_once = min(kQuads, int((kPart * 16 + 0.5f) * inv));  // quads
        const int mine = int((float(item) + 0.5f) * (0.25f * inv));
        const int mg = int((float(item - mine * lanes) + 0.5f) * inv), mc = item - mine * lanes - mg * rows;
        if (l < 16) {
            lds.stat[0][w][l] = wave.M[t];
            lds.stat[1][w][l] = wave.sum[t];
        }
        for (int q0 = 0; q0 < kQuads; q0 += at_once) {
            if (q0) __syncthreads();
            if (c < rows) {
                f32x4_t* at = lds.quad + w * lanes + g * rows + c;
                if (at_once == kQuads) {
#pragma unroll
                    for (int q = 0; q < kQuads; ++q) at[q * (NW * lanes)] = wave.o[t][q >> 2][q & 3];
                } else {
#pragma unroll
                    for (int q = 0; q < kQuads; ++q)
                        if (q >= q0 && q < q0 + at_once) at[(q - q0) * (NW * lanes)] = wave.o[t][q >> 2][q & 3];
                }
            }
            __syncthreads();
            if (mine < at_once && q0 + mine < kQuads) {
                // (four waves' results under way at a time, or each read would
                // wait for the one before)
                float by[NW], top = -INFINITY, total = 0.0f;
#pragma unroll
                for (int k = 0; k < NW; ++k) {
                    by[k] = lds.stat[0][k][mc];
                    top = fmaxf(top, by[k]);
                }
                const float m = top == -INFINITY ? 0.0f : top;
                f32x4_t v = {0.f, 0.f, 0.f, 0.f};
                const f32x4_t* from = lds.quad + mine * (NW * lanes) + item - mine * lanes;
#pragma unroll
                for (int k0 = 0; k0 < NW; k0 += 4) {
                    f32x4_t y[4];
                    float sum[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[k] = from[(k0 + k) * lanes];
                        sum[k] = lds.stat[1][k0 + k][mc];
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = exp2f_(by[k0 + k] - m);
                        total = __builtin_fmaf(f, sum[k], total);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(f, y[k][i], v[i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                out(q0 + mine, mg * 16 + mc, v, top, total);
            }
        }
    }
};

// The table of level pairs, filled by the whole workgroup.  (The levels come
// with the kernel's arguments: loads would wait for those of the first tiles.)
template <int NW>
__device__ __forceinline__ void fill_table(char* table, const uint32_t (&levels)[8]) {
    const int tid = threadIdx.x, copy = tid & 15;  // four lanes' copies
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int low = (tid >> 4) & 15;  // the low nibble of the thread's entries
    uint32_t pair = levels[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) pair = (low >> 1) == i ? levels[i] : pair;
    const uint32_t second = (low & 1 ? pair >> 16 : pair & 0xffffu) << 16;
#pragma unroll
    for (int e0 = 0; e0 < 256; e0 += 4 * NW) {
        const int high = (e0 + 4 * w) >> 4;  // (one for the wave)
        if (256 % (4 * NW) && high >= 16) break;
        const uint32_t v = ((levels[high >> 1] >> (16 * (high & 1))) & 0xffffu) | second;
        reinterpret_cast<u32x4_t*>(table)[(e0 + (tid >> 4)) * 16 + copy] = u32x4_t{v, v, v, v};
    }
}

// The first request's first row of q, and the one past the last request's last.
// Read at the start of a kernel, together with the lengths of its first unit (keep()
// stands where those are waited for): read when zero_rest() needs them they
// would be one more trip to memory at the end, 0.3 us of a call's 8.6.
struct Ends {
    int lo, hi;
    __device__ __forceinline__ explicit Ends(const Params& p) {
        typedef const __attribute__((address_space(4))) int32_t constant_t;
        constant_t* cu = (constant_t*)(uintptr_t)p.a.cu_q;
        lo = cu[0];
        hi = cu[p.a.batch];
    }
    __device__ __forceinline__ void keep() const { asm volatile("" ::"s"(lo), "s"(hi)); }
};

// Zeros, where the caller wants them, in the rows of the workgroup's head that are
// no request's, and in those past a request's max_q.  The workgroups of a head
// share the rows out; each comes here when its own work is done, and finds
// nothing in most calls.
template <int D>
__device__ __forceinline__ void zero_rest(const Params& p, const Ends& ends) {
    if (!p.zero_rest) return;
    const int index = p.by_heads.of(blockIdx.x), head = blockIdx.x - index * p.n_heads;
    const int count = p.by_heads.of(gridDim.x), threads = int(blockDim.x), tid = int(threadIdx.x);
    const int total = int(p.a.total_q), quads = p.group * (D / 8);
    auto zero = [&](int row, int quad) {
        *reinterpret_cast<u32x4_t*>(p.a.out + int64_t(row) * p.a.out_stride + int64_t(head) * p.group * D + 8 * quad) =
            u32x4_t{0u, 0u, 0u, 0u};
    };
    const int lo = min(max(ends.lo, 0), total), hi = min(max(ends.hi, lo), total);
    const int64_t rest = int64_t(lo + total - hi) * quads;
    for (int64_t i = int64_t(index) * threads + tid; i < rest; i += int64_t(count) * threads) {
        const int row = int(i / quads);
        zero(row < lo ? row : row - lo + hi, int(i - int64_t(row) * quads));
    }
    if (total <= p.a.max_q) return;
    const int l = tid & 63;
    for (int64_t r0 = int64_t(index) * threads + tid - l; r0 < p.a.batch; r0 += int64_t(count) * threads) {
        int from = 0, end = 0;
        if (r0 + l < p.a.batch) {
            from = min(max(p.a.cu_q[r0 + l], 0), total);
            end = min(max(p.a.cu_q[r0 + l + 1], from), total);
            from += min(end - from, p.a.max_q);
        }
        for (uint64_t some = __ballot(from < end); some; some &= some - 1) {
            const int who = __builtin_ctzll(some);
            const int a = __builtin_amdgcn_readlane(from, who), b = __builtin_amdgcn_readlane(end, who);
            for (int row = a; row < b; ++row)
                for (int quad = l; quad < quads; quad += 64) zero(row, quad);
        }
    }
}

constexpr size_t kTableBytes = 256 * 64 * 4;

constexpr int kWavesMany = 8;  // of a workgroup

// What a unit costs a workgroup beside its tiles, in tiles.
constexpr int kUnitCost = 16;

// A partial result: its quads, then M and the sum of each of its 16 rows.
__host__ __device__ constexpr int part_floats(int D) { return D / 16 * 64 * 4 + 32; }

// Waves of a workgroup, and of a SIMD: with 64 elements a wave fits 128
// registers and two workgroups share a CU, so that one's memory latencies
// overlap with the other's work; with 128 and 256 elements, and two tiles of
// rows, one workgroup of as many waves as the registers allow.
__host__ __device__ constexpr int waves_few(int D, int nt) { return D == 128 && nt == 1 ? 12 : D == 64 && nt == 2 ? 12 : 8; }
__host__ __device__ constexpr int simd_waves(int D, int nt) { return D == 64 && nt == 1 ? 4 : waves_few(D, nt) / 4; }
__host__ __device__ constexpr int groups_of_cu(int D, int nt) { return simd_waves(D, nt) * 4 / waves_few(D, nt); }

// Few rows: the NW waves of a workgroup take turns at the tiles of a unit's
// 16 * NT rows.
//
// With p.shares == 0 a workgroup has every p.step-th unit.  Otherwise the units'
// tiles (and kUnitCost more for each) are laid end to end and cut into p.shares
// equal shares, so that requests of any lengths occupy every CU to the end; a
// workgroup walks through the units of its share, writes the results of those
// that lie wholly inside it, and leaves its part of the first and the last to
// k_join_few.  The next unit's first loads are under way while the waves join.
//
// Bound, per 32 tokens and 16 rows of 128 elements: 4.4 KB of memory and 310
// vector instructions, 64 of them addresses of lookups.  On long runs of tokens
// the loop moves 5.3 to 5.9 TB/s, the rate of a large copy; what a call costs
// beside that is its first three memory trips (lengths, pages, tiles: 4 us),
// the uneven end and k_join_few.  At 64 elements a head, half the memory for
// almost as many instructions, it moves 3.3 TB/s.  With 8 cache heads of 128
// elements: 64 requests of 500 to 4096 tokens 44 us (122 MB), two of 90001 and
// 131071 tokens 59 us (241 MB, 4.1 TB/s), one of 301 tokens 9 us; 16 requests
// with 64 heads of 64 and a window of 1024 tokens 26.6 us (70 MB).
template <int D, int NT, int NW>
__device__ __forceinline__ void few(const Params& p, const Ends& ends) {
    using W = Wave<D, NT>;
    constexpr int kRows = 16 * NT;
    __shared__ struct {
        char table[kTableBytes];  // first: a looked-up byte's address needs no base added
        typename Join<D, NT, NW>::Lds join;
        u32x4_t qs[2][NT][W::NB][2][64];  // of the part at hand and the next
        float fs[2][NT][64];
        int scan[NW];
        int start[2];  // the share's first unit, and where it begins
    } sm;

    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const int share = p.by_heads.of(blockIdx.x), head = blockIdx.x - share * p.n_heads;
    const int units = p.a.batch * p.row_blocks;
    const int cost = p.shares ? kUnitCost : 0;
    int u = share;  // the unit at hand, and where it begins (in tiles; all fit 31 bits)
    int base = 0, from = 0, to = 0x7fffffff, size = to;
    const bool few_units = p.shares && units <= 64;
    Lengths known = {0, 0, 0};  // few_units: lane u's are those of unit u
    if (p.shares) {
        auto weight = [&](const Unit& x) { return x.empty ? 0 : x.tiles.count() + kUnitCost; };
        auto cost_of = [&](int i) { return weight(unit_of<false>(p, i, kRows)); };
        auto wave_sums = [&](int v) {  // (lanes before the first add 0)
            v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // 1, 2, 4, 8 lanes back in a row of 16
            v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
            v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
            v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
            v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // a row's last lane to rows 1 and 3
            v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
            return v;
        };
        auto cut = [&](int total) {
            // (a share of fewer tiles than two steps would not be worth its own workgroup)
            size = max((total + p.shares - 1) / p.shares, 2 * NW + kUnitCost);
            from = min(share * int64_t(size), int64_t(total));
            to = min(from + size, total);
        };
        // (k_join_few looks at every share: by default none of its units goes on)
        if (tid == 0) p.cuts[int64_t(share) * p.n_heads + head].x = -1;
        if (few_units) {  // every wave for itself
            const int request = p.by_row_blocks.of(min(l, units - 1));
            known = lengths_of<false>(p, request);
            const int mine = l < units ? weight(unit_of(p, l, kRows, request, known)) : 0;
            const int up = wave_sums(mine);
            cut(__builtin_amdgcn_readlane(up, 63));
            if (from >= to) return;
            const uint64_t here = __ballot(from >= up - mine && from < up);
            u = __builtin_ctzll(here);
            base = __builtin_amdgcn_readlane(up - mine, u);
        } else {
            const int per = (units + 64 * NW - 1) / (64 * NW);
            const int u0 = min(tid * per, units), u1 = min(u0 + per, units);
            int mine = 0;
            for (int i = u0; i < u1; ++i) mine += cost_of(i);
            int up = wave_sums(mine);
            if (l == 63) sm.scan[w] = up;
            __syncthreads();
            int total = 0;
            up -= mine;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const int v = sm.scan[i];
                up += i < w ? v : 0;
                total += v;
            }
            cut(total);
            if (from >= to) return;
            if (from >= up && from < up + mine) {
                int i = u0;
                for (; i + 1 < u1; ++i) {
                    const int v = cost_of(i);
                    if (from < up + v) break;
                    up += v;
                }
                sm.start[0] = i;
                sm.start[1] = up;
            }
            __syncthreads();
            u = __builtin_amdgcn_readfirstlane(sm.start[0]);
            base = __builtin_amdgcn_readfirstlane(sm.start[1]);
        }
    }

    // A unit and this share's tiles [lo, hi) of its n.  A unit without tiles,
    // whose rows see nothing, belongs to the share with the end of its cost.
    struct Part {
        Unit x;
        int base, lo, hi, n;
        bool any;
    };
    auto find = [&]() {
        Part f;
        f.any = false;
        while (u < units && base < to) {
            const int request = p.by_row_blocks.of(u);
            f.x = unit_of(p, u, kRows, request,
                          few_units ? Lengths{__builtin_amdgcn_readlane(known.c0, u), __builtin_amdgcn_readlane(known.c1, u),
                                              __builtin_amdgcn_readlane(known.have, u)}
                                    : lengths_of<true>(p, request));
            f.n = f.x.tiles.count();
            f.base = base;
            f.lo = min(max(from - base - cost, 0), f.n);
            f.hi = min(max(to - base - cost, 0), f.n);
            f.any = !f.x.empty && (f.n > 0 ? f.lo < f.hi : !p.shares || (base + cost > from && base + cost <= to));
            u += p.step;
            if (p.shares && !f.x.empty) base += f.n + cost;
            if (f.any) break;
        }
        return f;
    };

    W wave(p, sm.table, sm.qs[0], head);
    auto stage = [&](const Part& f, int side) {
        typename W::Row q;
        W::load_row(p, f.x, f.x.row0 + 16 * w + (l & 15), head, q);
        sm.fs[side][w][l] = W::stage_row(p, q, [&](int n, int s, const u32x4_t& v) { sm.qs[side][w][n][s][l] = v; });
    };
    Part now = find();
    ends.keep();
    if (!now.any) return;
    wave.read_ids(now.x, now.lo + w, now.hi, NW, wave.ids);
    if (w < NT) stage(now, 0);
    fill_table<NW>(sm.table, p.levels);
    wave.begin(now.x, now.lo + w, now.hi);
    for (int side = 0;; side ^= 1) {
        __syncthreads();
        // what the next part needs first is fetched now; its tiles while the
        // waves join
        const Part next = find();
        uint32_t next_ids[2] = {0u, 0u};
        if (next.any) {
            wave.read_ids(next.x, next.lo + w, next.hi, NW, next_ids);
            if (w < NT) stage(next, side ^ 1);
        }
        wave.qs = sm.qs[side];
#pragma unroll
        for (int t = 0; t < NT; ++t) wave.f[t] = sm.fs[side][t][l];
        wave.place(now.x, now.x.row0);
        wave.clear();
        wave.run(now.x, now.lo + w, now.hi, NW);
        wave.close();
        if (next.any) {
            wave.ids[0] = next_ids[0], wave.ids[1] = next_ids[1];
            wave.begin(next.x, next.lo + w, next.hi);
        }
        const bool all = now.lo == 0 && now.hi == now.n;
        float* part = p.part + ((int64_t(share) * p.n_heads + head) * 2 + (now.lo == 0 ? 1 : 0)) * NT * part_floats(D);
        if (now.lo == 0 && !all && tid == 0)
            p.cuts[int64_t(share) * p.n_heads + head] =
                make_int4((now.base + cost + now.n - 1) / size, now.x.q0, now.x.rows, now.x.row0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t) __syncthreads();
            const int rows = min(now.x.rows - now.x.row0 - 16 * t, 16);
            if (rows <= 0) break;
            Join<D, NT, NW>::run(wave, t, rows, w, sm.join, [&](int quad, int lane, f32x4_t v, float top, float total) {
                if (all) {
                    store_quad<D>(p, now.x.q0, now.x.rows, head, now.x.row0 + 16 * t + (lane & 15), quad, lane >> 4, v, total);
                    return;
                }
                float* at = part + t * part_floats(D);
                reinterpret_cast<f32x4_t*>(at)[quad * 64 + lane] = v;
                if (quad == 0 && lane < 16) {
                    at[D / 16 * 256 + lane] = top;
                    at[D / 16 * 256 + 16 + lane] = total;
                }
            });
        }
        if (!next.any) return;
        now = next;
    }
}

template <int D, int NT, int NW>
__global__ __launch_bounds__(64 * NW, simd_waves(D, NT)) void k_attn_few(Params p) {
    const Ends ends(p);
    few<D, NT, NW>(p, ends);
    zero_rest<D>(p, ends);
}

// Few rows and units for most of the GPU's waves: each wave has units of its own,
// alone.  A workgroup has every p.step-th unit, and its waves take the next one as
// they come free (counted in LDS), so that lengths even out; which wave has a unit
// does not change its result.  What a wave waits for between units is covered by
// the others; asking for the next one ahead was slower, because it is then with
// the wrong wave (1000 requests of 16 to 1536 tokens: 200 us, 139 so).
//
// Bound by the same instructions a tile as k_attn_few, but without its 5 us a unit
// and workgroup: 384 requests of 400 to 500 tokens, 8 cache heads of 128 elements,
// 48 us (188 MB, 3.9 TB/s), 99 us there; 512 with heads of 64 36 us, 64 there.
template <int D, int NT, int NW>
__device__ __forceinline__ void alone(const Params& p, const Ends& ends) {
    using W = Wave<D, NT>;
    constexpr int kRows = 16 * NT;
    __shared__ struct {
        char table[kTableBytes];
        u32x4_t qs[NW][NT][W::NB][2][64];
        int taken;  // units of the workgroup's
    } sm;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const int group = p.by_heads.of(blockIdx.x), head = blockIdx.x - group * p.n_heads;
    const int units = p.a.batch * p.row_blocks;
    if (threadIdx.x == 0) sm.taken = NW;  // (the first ones are each wave's own)
    fill_table<NW>(sm.table, p.levels);
    __syncthreads();
    W wave(p, sm.table, sm.qs[w], head);
    for (int k = w;;) {
        const int u = group + k * p.step;
        if (u >= units) return;
        const Unit x = unit_of<true>(p, u, kRows);
        ends.keep();
        if (!x.empty) {
            const int tiles = x.tiles.count();
            wave.read_ids(x, 0, tiles, 1, wave.ids);
            typename W::Row q[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) W::load_row(p, x, x.row0 + 16 * t + (l & 15), head, q[t]);
            wave.begin(x, 0, tiles);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                wave.f[t] = W::stage_row(p, q[t], [&](int n, int s, const u32x4_t& v) { sm.qs[w][t][n][s][l] = v; });
            wave.place(x, x.row0);
            wave.clear();
            wave.run(x, 0, tiles, 1);
            wave.close();
#pragma unroll
            for (int t = 0; t < NT; ++t) wave.write(x, x.row0, t);
        }
        if (l == 0) k = __hip_atomic_fetch_add(&sm.taken, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        k = __builtin_amdgcn_readfirstlane(k);
    }
}

template <int D, int NT, int NW>
__global__ __launch_bounds__(64 * NW) void k_attn_alone(Params p) {
    const Ends ends(p);
    alone<D, NT, NW>(p, ends);
    zero_rest<D>(p, ends);
}

// Results of 16 rows added up over the workgroups that have them; a thread has
// one quad of one lane.  A call's last launch is bound by its memory trips (4 us
// for 256 units of two results, 2.5 us of them an empty launch), so several
// results are under way at a time.
template <int D>
struct Total {
    float top = -INFINITY, total = 0.0f;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};

    template <int K>
    struct Some {
        float M[K], sum[K];
        f32x4_t y[K];
        // at(k): result k
        template <typename At>
        __device__ __forceinline__ void load(At at) {
            const int quad = threadIdx.x >> 6, l = threadIdx.x & 63, c = l & 15;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float* from = at(k);
                M[k] = from[D / 16 * 256 + c];
                sum[k] = from[D / 16 * 256 + 16 + c];
                y[k] = reinterpret_cast<const f32x4_t*>(from)[quad * 64 + l];
            }
        }
    };

    // the first n (1 or more) of some results
    template <int K>
    __device__ __forceinline__ void add(const Some<K>& r, int n) {
        float next = top;
#pragma unroll
        for (int k = 0; k < K; ++k) next = k < n ? fmaxf(next, r.M[k]) : next;
        const float m = next == -INFINITY ? 0.0f : next;
        const float was = exp2f_(top - m);
        total *= was;
        v *= was;
        top = next;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float by = k < n ? exp2f_(r.M[k] - m) : 0.0f;
            total = k < n ? __builtin_fmaf(by, r.sum[k], total) : total;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = k < n ? __builtin_fmaf(by, r.y[k][i], v[i]) : v[i];
        }
    }

    __device__ __forceinline__ void store(const Params& p, int q0, int rows, int row0, int head) const {
        const int l = threadIdx.x & 63;
        store_quad<D>(p, q0, rows, head, row0 + (l & 15), threadIdx.x >> 6, l >> 4, v, total);
    }
};

// The results of a unit whose tiles lie in several shares, by the first of them.
// Its own and the next share's are read before it is known whether there is
// such a unit.
template <int D, int NT>
__global__ __launch_bounds__(D * 4) void k_join_few(Params p) {
    const int first = p.by_heads.of(blockIdx.x), head = blockIdx.x - first * p.n_heads;
    auto at = [&](int s, int t) {
        return p.part + (((int64_t(s) * p.n_heads + head) * 2 + (s == first ? 1 : 0)) * NT + t) * part_floats(D);
    };
    typename Total<D>::template Some<2> two;
    two.load([&](int k) { return at(min(first + k, p.shares - 1), 0); });
    __builtin_amdgcn_sched_barrier(0);
    const int4 cut = p.cuts[blockIdx.x];
    if (cut.x < 0) return;
    for (int t = 0; t < NT; ++t) {
        if (t) two.load([&](int k) { return at(min(first + k, cut.x), t); });
        Total<D> sum;
        sum.add(two, cut.x - first + 1);
        for (int s = first + 2; s <= cut.x; s += 8) {
            typename Total<D>::template Some<8> more;
            more.load([&](int k) { return at(min(s + k, cut.x), t); });
            sum.add(more, cut.x - s + 1);
        }
        sum.store(p, cut.y, cut.z, cut.w + 16 * t, head);
    }
}

// The results of a block whose tiles were split, 16 rows a workgroup.
template <int D, int NT>
__global__ __launch_bounds__(D * 4) void k_join_many(Params p) {
    constexpr int kTiles = kWavesMany * NT;
    const int u = blockIdx.x / kTiles, t = blockIdx.x % kTiles;
    const int by = p.by_heads.of(u), head = u - by * p.n_heads;
    const Unit x = unit_of<true>(p, by, 16 * kTiles);
    const int row0 = x.row0 + 16 * t;
    if (row0 >= x.rows) return;
    Total<D> sum;
    for (int s = 0; s < p.splits; s += 8) {
        typename Total<D>::template Some<8> some;
        some.load([&](int k) {
            const int64_t part = int64_t(by) * p.splits + min(s + k, p.splits - 1);
            return p.part + ((part * p.n_heads + head) * kTiles + t) * part_floats(D);
        });
        sum.add(some, p.splits - s);
    }
    sum.store(p, x.q0, x.rows, row0, head);
}

// Many rows: every wave has 16 * NT rows of its own.  The workgroup's waves
// turn the codes into operands together, each a part of the next 8192 / D
// tokens (a frame), and read from LDS those of the present one: looked up by
// every wave for itself, they were a third of all instructions (two prompt
// chunks of 2048 queries over 5000 to 6144 tokens, 32 heads on 8 of 128
// elements: 627 us by every wave, 490 us so).
//
// p.splits workgroups share the tiles of a block of rows; with more than one
// each leaves a partial result to k_join_many.
//
// Bound: per 32 rows and 32 tokens of 128 elements 32 matrix instructions, 512
// cycles, and 187 vector instructions, 860 cycles with the exponentials: 16
// weights a lane at 9 instructions, their maximum, sums and scales.  Two waves
// a SIMD keep the vector units at 58 % and the matrix units at 31 %; registers
// allow no third.  The chunks above take 392 us, 780 TFLOP/s, against 243 us of
// the two products at a large library product's rate.  Slower by measurement:
// the next tile's products in the same wave beside the weights of this one
// (455 us), waves 4-7 a barrier behind waves 0-3 so that one of a SIMD
// multiplies while the other weighs (532 us), a higher priority of the waves
// that multiply (456 us).
template <int D>
struct Frame {
    static constexpr int T = 8192 / D, NB = D / 64;
    u32x4_t k[16][64];  // of half tile h, block n, step s: [2 * (h * NB + n) + s]
    u32x4_t v[16][64];  // of tile j, block n, element i: [4 * (j * NB + n) + i]
    float ks[NB][T], vs[NB][T], e[T];  // absmax; exponent of the values' largest
};

template <int D, int NT>
__device__ __forceinline__ void many(const Params& p, const Ends& ends) {
    using W = Wave<D, NT>;
    using F = Frame<D>;
    constexpr int NW = kWavesMany, T = F::T, NB = F::NB, HT = T / 16;  // HT: half tiles of a frame
    static_assert(NW == 8, "what each wave turns into operands");
    __shared__ struct {
        char table[kTableBytes];
        F frames[2];
    } sm;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    // neighbouring workgroups are on different XCDs and take different heads,
    // so with 8 heads an XCD's L2 holds one
    const int bys = p.by_heads.of(blockIdx.x), head = blockIdx.x - bys * p.n_heads;
    const int by = p.by_splits.of(bys), split = bys - by * p.splits;
    Unit x = unit_of<true, T>(p, by, 16 * NT * NW);
    ends.keep();
    if (x.empty) return;
    x.row0 += w * 16 * NT;
    const bool idle = x.row0 >= x.rows;  // a wave without rows, which only helps
    W wave(p, sm.table, nullptr, head);
    u32x4_t qs[NT][NB][2];
    typename W::Row q[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) W::load_row(p, x, x.row0 + 16 * t + (l & 15), head, q[t]);

    // this workgroup's frames of the list
    const int all = x.tiles.count();
    const int first = int(int64_t(all) * split / p.splits), last = int(int64_t(all) * (split + 1) / p.splits);
    const int count = last - first;
    auto frame_at = [&](int i) { return x.tiles.at(min(first + i, last - 1)); };

    // What the wave turns into operands of frame i: waves 0-3 two (half tile,
    // block) pairs of keys each, waves 4-7 one (tile, block) pair of the values;
    // waves 0 and 1 have the scales too, a lane two neighbouring ones.
    const bool values = w >= 4;
    const int32_t* row = p.a.table + int64_t(x.request) * p.a.width;
    uint32_t ids = 0;  // lane y: the page of half tile y, counted from frame 64 / HT * k on
    uint32_t raw[8], raw_scales = 0;
    uint32_t there = 0;  // bit h: the page of half tile h exists
    auto load = [&](int i) {
        const int at = (i % (64 / HT)) * HT;
        if (at == 0) {
            const int t = frame_at(i + l / HT) * HT + l % HT;
            ids = uint32_t(row[min(t >> (p.pshift - 4), max(p.a.width - 1, 0))]);
        }
        const int t0 = __builtin_amdgcn_readfirstlane(frame_at(i)) * T;
        there = uint32_t(__ballot(ids < p.n_pages) >> at) & ((1u << HT) - 1);
        auto entry = [&](int h) { return wave.entry(uint32_t(__builtin_amdgcn_readlane(int(ids), at + h)), t0 + 16 * h); };
        if (!values) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = (2 * w + k) / NB, n = (2 * w + k) % NB;
                const auto r = W::buffer(p.codes[0] + entry(h) * (D / 2), 16 * (D / 2));
                const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, wave.key_at + 32 * n, 0, 0);
                raw[2 * k] = v[0], raw[2 * k + 1] = v[1];
            }
            if (w < 2) {
                const int h = l / (8 * NB);
                const int64_t at0 = wave.entry(uint32_t(__shfl(int(ids), at + h)), t0 + 16 * h) * NB;
                raw_scales = *reinterpret_cast<const uint32_t*>(p.scales[w] + at0 + 2 * (l % (8 * NB)));
            }
        } else {
            const int n = (w - 4) % NB;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const auto r = W::buffer(p.codes[1] + entry(2 * ((w - 4) / NB) + h) * (D / 2), 16 * (D / 2));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    raw[4 * h + j] = __builtin_amdgcn_raw_buffer_load_b16(r, wave.value_at + j * (D / 2) + 32 * n, 0, 0);
            }
        }
    };
    auto turn = [&](F& to) {
        u32x4_t ready[4];  // (all looked up before the first is written: a write would wait for the lookups before it)
        if (!values) {
#pragma unroll
            for (int k = 0; k < 4; ++k) ready[k] = wave.look_up(raw[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) to.k[4 * w + k][l] = ready[k];
            if (w < 2) {
                const float a = bf16_lo(raw_scales), b = bf16_hi(raw_scales);
                const int token = 2 * l / NB, n = 2 * l % NB;
                float(&dst)[NB][T] = w ? to.vs : to.ks;
                if constexpr (NB == 1) dst[0][token] = a, dst[0][token + 1] = b;
                else dst[n][token] = a, dst[n + 1][token] = b;
                if (w) {
                    if constexpr (NB == 1) {
                        to.e[token] = W::exponent_of(a), to.e[token + 1] = W::exponent_of(b);
                    } else {
                        float m = fmaxf(a, b);
                        if constexpr (NB == 4) m = fmaxf(m, __shfl_xor(m, 1, 64));
                        to.e[token] = W::exponent_of(m);
                    }
                }
            }
        } else {
            wave.turn_values(raw, [&](int i, const u32x4_t& a) { ready[i] = a; });
#pragma unroll
            for (int k = 0; k < 4; ++k) to.v[4 * (w - 4) + k][l] = ready[k];
        }
    };

    if (count > 0) load(0);
    fill_table<NW>(sm.table, p.levels);
#pragma unroll
    for (int t = 0; t < NT; ++t)
        wave.f[t] = W::stage_row(p, q[t], [&](int n, int s, const u32x4_t& v) { qs[t][n][s] = v; });
    wave.place(x, x.row0);
    wave.clear();
    __syncthreads();
    uint32_t there_now = there, there_next = 0;
    if (count > 0) {
        turn(sm.frames[0]);
        if (count > 1) load(1), there_next = there;
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) {
        const F& f = sm.frames[i & 1];
        const int t0 = __builtin_amdgcn_readfirstlane(frame_at(i)) * (T / kTile);
#pragma unroll
        for (int j = 0; j < T / kTile; ++j) {
            const int tile = t0 + j, token = tile * kTile;
            if (idle || token > wave.pos_last) continue;
            if (p.a.window && token + kTile - 1 <= wave.before_window(wave.pos_first) && token >= p.a.sinks) continue;
            auto four = [&](const float* from, int h) {
                return *reinterpret_cast<const f32x4_t*>(from + kTile * j + 16 * h + 4 * wave.g);
            };
            // Operands are read a step ahead of the products that need them: the
            // compiler by itself has each wait for its own.  (sched_barrier: nothing
            // moves past)
            u32x4_t ka[2][NB];
            auto read_keys = [&](int step) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    ka[step & 1][n] = f.k[2 * ((2 * j + (step >> 1)) * NB + n) + (step & 1)][l];
            };
            typename W::Products acc[2];
            f32x4_t ks[2][NB];
            read_keys(0);
            read_keys(1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int step = 0; step < 4; ++step) {
                W::multiply(ka[step & 1], [&](int t, int n) { return qs[t][n][step & 1]; }, step & 1, acc[step >> 1]);
                if (step < 2) {
                    read_keys(step + 2);
                } else {
#pragma unroll
                    for (int n = 0; n < NB; ++n) ks[step - 2][n] = four(f.ks[n], step - 2);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            f32x4_t vs[2][NB], e[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int n = 0; n < NB; ++n) vs[h][n] = four(f.vs[n], h);
                e[h] = four(f.e, h);
            }
            float s2[NT][2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) W::add_up(acc[h], [&](int r, int n) { return ks[h][n][r]; }, h, s2);
            const bool here[2] = {(there_now >> (2 * j) & 1) != 0, (there_now >> (2 * j + 1) & 1) != 0};
            if (!wave.whole(tile, here)) wave.hide(tile, here, s2);
            u32x4_t wt[NT][NB];
            wave.weigh([&](int h, int r, int n) { return vs[h][n][r]; }, [&](int h, int r) { return e[h][r]; }, s2, wt);
            u32x4_t va[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) va[k] = f.v[4 * j * NB + k][l];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const u32x4_t a = va[k];
                    if (n + 1 < NB) va[k] = f.v[4 * (j * NB + n + 1) + k][l];
#pragma unroll
                    for (int t = 0; t < NT; ++t) wave.o[t][n][k] = mfma_f16(a, wt[t][n], wave.o[t][n][k]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        if (i + 1 < count) turn(sm.frames[(i + 1) & 1]);
        if (i + 2 < count) load(i + 2);
        there_now = there_next, there_next = there;
        __syncthreads();
    }
    if (idle) return;
    wave.close();
    if (p.splits == 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) wave.write(x, x.row0, t);
        return;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float* at = p.part + ((int64_t(bys) * p.n_heads + head) * (NW * NT) + w * NT + t) * part_floats(D);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<f32x4_t*>(at)[(4 * n + i) * 64 + l] = wave.o[t][n][i];
        if (l < 16) {
            at[D / 16 * 256 + l] = wave.M[t];
            at[D / 16 * 256 + 16 + l] = wave.sum[t];
        }
    }
}

template <int D, int NT>
__global__ __launch_bounds__(64 * kWavesMany) void k_attn_many(Params p) {
    const Ends ends(p);
    many<D, NT>(p, ends);
    zero_rest<D>(p, ends);
}

// Every row's output of a call that computes none.
__global__ __launch_bounds__(256) void k_zero(uint16_t* out, int64_t stride, int64_t rows, int quads) {
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < rows * quads; i += gridDim.x * int64_t(256)) {
        const int64_t row = i / quads;
        *reinterpret_cast<u32x4_t*>(out + row * stride + 8 * (i - row * quads)) = u32x4_t{0u, 0u, 0u, 0u};
    }
}

// How a call is cut up.
struct Cut {
    bool many;
    bool alone;
    int nt, row_blocks, shares, splits;
};

constexpr int most_tiles(int D) { return D == 256 ? 1 : 2; }  // of rows, a wave

Cut cut_of(int D, int n_heads, const kv::Attn& a) {
    Cut c;
    const int group = a.q_heads / n_heads;
    const int64_t rows = int64_t(a.max_q) * group;
    int64_t tokens = a.max_len;
    if (a.window) tokens = std::min<int64_t>(tokens, int64_t(a.window) + std::min(a.sinks, a.max_len) + rows / group + 64);
    const int64_t tiles = kv::cdiv(tokens, kTile) + 2;
    c.nt = rows > 16 ? most_tiles(D) : 1;
    c.row_blocks = int(kv::cdiv(rows, 16 * c.nt));
    const int64_t units = std::min<int64_t>(int64_t(a.batch) * c.row_blocks, 0x7fffffff);
    // Many: the codes are turned into operands once for 256 rows, and not once for
    // 32, but a workgroup does not fill up with fewer rows, and its partial results
    // are as large as 256 rows.  That pays from 96 rows on (8 cache heads of 128
    // elements, 32 requests of 2048 tokens, us: 64 rows 77 against 53, 128 rows 81
    // against 107, 512 rows 195 against 390), and if there is work of 128 tiles
    // for each CU (1 request of 2048 tokens: 512 rows 37 against 27; of 32768: 128
    // rows 53 against 56, 512 rows 110 against 165).
    c.many = rows >= 96 && units * tiles > 256 * 128 / n_heads;
    c.shares = 0, c.splits = 1;
    const int64_t at_once = 256 * groups_of_cu(D, c.nt);  // workgroups of few rows
    // Alone: units for three of five waves, and none so long that the GPU would wait
    // for it (us in k_attn_few and alone, 8 cache heads of 128: 192 requests of 16
    // to 500 tokens 38 and 31, 128 of them 27 and 32; 256 of 100 to 2000 90 and 108,
    // 384 of them 122 and 114; 384 of 1900 to 2000 223 and 184; 384 of 300 to 3000,
    // heads of 256, 274 and 318).
    const int64_t waves = at_once * waves_few(D, c.nt), all = units * n_heads;
    c.alone = !c.many && all * 5 >= waves * 3 && tokens <= 2048 && tokens * waves <= all * 2048;
    if (c.many) {
        c.row_blocks = int(kv::cdiv(rows, 16 * c.nt * kWavesMany));
        // A workgroup occupies a CU.  With less than two blocks for three CUs the
        // blocks' tokens are split, as far as 512 tokens take longer than a partial
        // result and its share of the join (192 rows of 1 request of 32768 tokens:
        // 1286 us in 8 workgroups, 64 us in 256; of 2048 tokens: 84 and 33).
        const int64_t blocks = int64_t(a.batch) * c.row_blocks * n_heads;
        if (blocks <= 170) c.splits = int(std::max<int64_t>(std::min(256 / blocks, tokens / 512), 1));
    } else if (!c.alone) {
        // Six steps of every wave take about as long as a second launch (1 request,
        // whole and shared, us: 128 elements a head, 2048 tokens 16.5 and 16.1, 3000
        // tokens 21.6 and 17.0; 256 elements, 1536 tokens 23.7 and 23.6, 2048 tokens
        // 29.0 and 23.6; 64 elements, 1536 tokens 12.1 and 13.7, 2048 tokens 14.3 and
        // 14.0).  The more of the GPU one request's blocks of equal length fill, the
        // less there is to win (512 queries, 8 heads of 256, 2048 tokens: 34.4 and
        // 43.5).  Requests of different lengths are shared however many they are (64
        // of 40 to 16384 tokens, 8 heads of 128: 117 and 64; of 400 to 4096: 45.6 and
        // 38.6), but those that fill the GPU by themselves from eight steps on (32 of
        // 1800 to 2048 tokens, 24 rows: 28.8 and 37.1).
        const int64_t filled = std::min(int64_t(c.row_blocks) * n_heads, at_once);
        const int64_t steps = units < at_once / n_heads ? 6 : 8;
        // (a share's end has to fit 31 bits too: at most a tile for each share past the last)
        if (tokens * (at_once - filled) > steps * waves_few(D, c.nt) * kTile * at_once &&
            units * (tiles + kUnitCost) < 0x7fffffff - 1024)
            c.shares = int(std::max<int64_t>(at_once / n_heads, 1));
    }
    return c;
}

size_t part_bytes(int D, int n_heads, int batch, const Cut& c) {
    const size_t each = size_t(n_heads) * c.nt * part_floats(D) * 4;
    return c.many ? size_t(batch) * c.row_blocks * c.splits * kWavesMany * each : c.shares * 2 * each;
}

}  // namespace

namespace kv {

size_t attention_ws_bytes(const Cache& c, const Attn& a) {
    if (a.max_q == 0) return 0;
    const Cut k = cut_of(c.head_dim, c.n_heads, a);
    if (!k.shares && k.splits == 1) return 0;
    return part_bytes(c.head_dim, c.n_heads, a.batch, k) + size_t(k.shares) * c.n_heads * sizeof(int4);
}

template <int D, int NT>
static void launch_few(const Params& p, bool join, unsigned grid, hipStream_t st) {
    constexpr int NW = waves_few(D, NT);
    if (!join) hipLaunchKernelGGL((k_attn_few<D, NT, NW>), dim3(grid), dim3(64 * NW), 0, st, p);
    else hipLaunchKernelGGL((k_join_few<D, NT>), dim3(grid), dim3(D * 4), 0, st, p);
}

template <int D, int NT>
static void launch_alone(Params p, int64_t units, hipStream_t st) {
    constexpr int NW = waves_few(D, NT) * groups_of_cu(D, NT);  // of a CU
    const int per_head = int(std::min<int64_t>(cdiv(units, NW), std::max(256 / p.n_heads, 1)));
    p.step = per_head;
    hipLaunchKernelGGL((k_attn_alone<D, NT, NW>), dim3(unsigned(per_head * p.n_heads)), dim3(64 * NW), 0, st, p);
}

template <int D>
static int launch(const Cache& c, const Attn& a, bool zero_rest, void* ws, hipStream_t st) {
    constexpr int NT2 = most_tiles(D);
    const Cut k = cut_of(D, c.n_heads, a);
    const int64_t units = int64_t(a.batch) * k.row_blocks;
    // Blocks of many rows have a workgroup of 512 threads each, of less than 2^32
    // in a grid; few rows are walked through, where a wave's next unit, at most 8192
    // past the last, has to fit 31 bits.
    if (k.many ? units * c.n_heads > 0x7fffff : (units + 8192) * c.n_heads > 0x7fffffff) return NF4_EINVAL;
    Params p = {};
    for (int s = 0; s < 2; ++s) p.codes[s] = c.codes[s], p.scales[s] = c.scales[s];
    p.n_pages = uint32_t(c.n_pages);
    p.n_heads = c.n_heads, p.pshift = c.pshift, p.qt = c.qt;
    for (int i = 0; i < 8; ++i) p.levels[i] = level_f16(c.qt, 2 * i) | level_f16(c.qt, 2 * i + 1) << 16;
    p.a = a;
    p.zero_rest = zero_rest;
    p.group = a.q_heads / c.n_heads;
    p.row_blocks = k.row_blocks;
    p.by_group = kv::Div::by(p.group), p.by_row_blocks = kv::Div::by(p.row_blocks), p.by_heads = kv::Div::by(c.n_heads), p.by_splits = kv::Div::by(k.splits);
    p.shares = k.shares, p.splits = k.splits;
    p.part = static_cast<float*>(ws);
    p.cuts = reinterpret_cast<int4*>(static_cast<char*>(ws) + part_bytes(D, c.n_heads, a.batch, k));
    const unsigned all = unsigned(units * c.n_heads);
    if (k.many) {
        hipLaunchKernelGGL((k_attn_many<D, NT2>), dim3(all * k.splits), dim3(64 * kWavesMany), 0, st, p);
        if (k.splits == 1) return launch_status();
        if (const int rc = launch_status()) return rc;
        hipLaunchKernelGGL((k_join_many<D, NT2>), dim3(all * kWavesMany * NT2), dim3(D * 4), 0, st, p);
        return launch_status();
    }
    if (k.alone) {
        if (k.nt == 2) launch_alone<D, NT2>(p, units, st);
        else launch_alone<D, 1>(p, units, st);
        return launch_status();
    }
    // No more workgroups than run at a time, each with every so many-th unit: its
    // table serves them all, and the next unit's loads are under way early (64
    // requests of 100 to 2000 tokens, 8 heads of 128: 33 us by a workgroup each, 29.5).
    const int64_t at_once = std::max(256 * groups_of_cu(D, k.nt) / c.n_heads, 1);
    const int per_head = k.shares ? k.shares : int(std::min(units, at_once));
    p.step = k.shares ? 1 : per_head;
    const unsigned grid = unsigned(per_head * c.n_heads);
    for (int join = 0; join < (k.shares ? 2 : 1); ++join) {
        if (k.nt == 2) launch_few<D, NT2>(p, join, grid, st);
        else launch_few<D, 1>(p, join, grid, st);
        if (const int rc = launch_status()) return rc;
    }
    return NF4_OK;
}

int attention(const Cache& c, const Attn& a, bool zero_rest, void* ws, hipStream_t st) {
    if (a.max_q == 0) {
        if (!zero_rest) return NF4_OK;
        const int quads = a.q_heads * (c.head_dim / 8);
        const int64_t blocks = std::min<int64_t>(cdiv(a.total_q * quads, 256), 4096);
        hipLaunchKernelGGL(k_zero, dim3(unsigned(blocks)), dim3(256), 0, st, a.out, a.out_stride, a.total_q, quads);
        return launch_status();
    }
    return c.head_dim == 64 ? launch<64>(c, a, zero_rest, ws, st)
         : c.head_dim == 128 ? launch<128>(c, a, zero_rest, ws, st) : launch<256>(c, a, zero_rest, ws, st);
}

}  // namespace kv
