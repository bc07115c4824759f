// kv_device.h -- building blocks shared by the cache kernels (gfx950 only).
//
// These files are compiled with -ffp-contract=off: a product and a sum are
// fused only where __builtin_fmaf says so, because the rotation is defined
// with each operation rounded (see nf4kv.h).
#pragma once

#include "../nf4_device.h"
#include "nf4kv.h"

namespace kv {

// Records a failed launch for nf4_kv_last_hip_error(); NF4_OK or NF4_ELAUNCH.
int launch_status();

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The cache as the kernels see it (page_size = 1 << pshift).
struct Cache {
    uint8_t* codes[2];    // keys, values
    uint16_t* scales[2];
    int64_t n_pages;
    int n_heads, head_dim, pshift, qt;
};

struct Rope {  // rot == 0: no rotation
    const int32_t* positions;
    const float* table;
    int64_t max_pos;
    int rot, interleaved;
};

int plan(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* done, int batch, int32_t* table, int width,
         int pshift, int32_t* ring, int capacity, const int32_t* state, int max_tokens, int32_t* lens_out,
         int32_t* cu, int64_t* slots, int32_t* positions, int32_t* free_out, int32_t* refused, hipStream_t st);
int rope_table(float* table, int64_t max_pos, int rot, float base, const nf4_rope_scaling& s, hipStream_t st);
int rope(const void* x, int64_t xt, int64_t xh, void* y, int64_t yt, int64_t yh, int64_t tokens, int heads, int dim,
         bool bf16, const Rope& r, float sign, hipStream_t st);
int append(const Cache& c, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
           const int64_t* slots, int64_t tokens, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
           int64_t q_out_stride, int q_heads, const Rope& r, hipStream_t st);
int read(const Cache& c, const int64_t* slots, int64_t tokens, uint16_t* k_out, uint16_t* v_out, hipStream_t st);

struct Attn {
    const uint16_t* q;
    int64_t q_stride, total_q;
    uint16_t* out;
    int64_t out_stride;
    const int32_t *cu_q, *kv_lens, *table;
    int width, batch, q_heads, max_q, max_len, window, sinks;
    float scale;
};
size_t attention_ws_bytes(const Cache& c, const Attn& a);
int attention(const Cache& c, const Attn& a, bool zero_rest, void* ws, hipStream_t st);


// Division of 0 <= n < 2^31 by a number fixed on the host, as a product: with
// 2^(l-1) < d <= 2^l and mul = ceil(2^(31+l) / d), n * mul / 2^(31+l) exceeds
// n / d by less than 1 / d.
struct Div {
    uint32_t mul;  // 0 for d == 1
    int shift;
    static Div by(uint32_t d) {
        int l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        return d == 1 ? Div{0, 0} : Div{uint32_t(((uint64_t(1) << (31 + l)) + d - 1) / d), l - 1};
    }
    __device__ __forceinline__ int of(int n) const { return mul ? int(__umulhi(uint32_t(n), mul) >> shift) : n; }
};

// ---- one rotated pair: each product and sum rounded by itself
struct Pair { float a, b; };
__device__ __forceinline__ Pair turn(float a, float b, float c, float s) {
    return {a * c - b * s, b * c + a * s};
}

// ---- bf16 in groups of 8 (16 bytes) or fewer
template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&v)[N]) {
    static_assert(N == 1 || N == 2 || N == 4 || N % 8 == 0, "group size");
    if constexpr (N == 1) {
        v[0] = nf4dev::bf16_f(p[0]);
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 2) w[0] = *reinterpret_cast<const uint32_t*>(p);
        if constexpr (N == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        if constexpr (N >= 8) {
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                const uint4 t = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
            }
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            v[2 * i] = nf4dev::bf16_lo(w[i]);
            v[2 * i + 1] = nf4dev::bf16_hi(w[i]);
        }
    }
}

template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        p[0] = nf4dev::to_bf16(v[0]);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = nf4dev::pack_bf16x2(v[2 * i], v[2 * i + 1]);
        if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
        if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        if constexpr (N >= 8) {
#pragma unroll
            for (int i = 0; i < N / 8; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
}

template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 t = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = p[i];
    }
}

template <int N>
__device__ __forceinline__ void store_f32(float* p, const float (&v)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = v[i];
    }
}

}  // namespace kv
