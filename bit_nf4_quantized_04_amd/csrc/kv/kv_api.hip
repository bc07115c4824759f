// kv_api.hip -- the extern "C" entry points declared in nf4kv.h: argument
// checks, then the launches.  No allocation, no synchronization.
#include <math.h>

#include "kv_device.h"

namespace {

thread_local int g_last_hip_error = 0;

inline bool bad(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

int log2_of(int v) {
    for (int s = 0; s < 31; ++s)
        if ((1 << s) == v) return s;
    return -1;
}

int page_shift(int page_size) {
    const int s = log2_of(page_size);
    return s >= 4 && s <= 8 ? s : -1;
}

int cache_of(const nf4_kv_cache* t, kv::Cache* c) {
    if (!t || bad(t->k_codes) || bad(t->v_codes) || bad(t->k_scales) || bad(t->v_scales)) return NF4_EINVAL;
    if (t->n_pages < 1 || t->n_pages > 0x7fffffff || t->n_heads < 1 || t->n_heads > 1024) return NF4_EINVAL;
    if (t->head_dim != 64 && t->head_dim != 128 && t->head_dim != 256) return NF4_EUNSUPPORTED;
    if (t->quant_type != NF4_QUANT_NF4 && t->quant_type != NF4_QUANT_FP4) return NF4_EUNSUPPORTED;
    *c = {{t->k_codes, t->v_codes}, {t->k_scales, t->v_scales}, t->n_pages, t->n_heads, t->head_dim,
          page_shift(t->page_size), t->quant_type};
    return c->pshift < 0 ? NF4_EUNSUPPORTED : NF4_OK;
}

// A token has more than one thread: more of them than this is more threads than a
// grid has, and the products that a launch makes of smaller numbers fit 64 bits.
constexpr int64_t kMostTokens = 0x7fffffff;

// A rotation of rot of head_dim elements; rot == 0 (where allowed) is none.
int rope_of(const int32_t* positions, const float* table, int64_t max_pos, int rot, int layout, int head_dim,
            bool may_be_none, kv::Rope* r) {
    *r = {positions, table, max_pos, rot, layout == NF4_ROPE_INTERLEAVED};
    if (rot == 0 && may_be_none) return NF4_OK;
    if (layout != NF4_ROPE_HALF && layout != NF4_ROPE_INTERLEAVED) return NF4_EUNSUPPORTED;
    if (rot < 2 || rot % 2 || rot > head_dim) return NF4_ESHAPE;
    if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3) || bad(table) || max_pos < 1) return NF4_EINVAL;
    return NF4_OK;
}

int rope_call(const void* x, int64_t xt, int64_t xh, void* y, int64_t yt, int64_t yh, int64_t tokens, int heads,
              int dim, int is_bf16, const int32_t* positions, const float* table, int64_t max_pos, int rot,
              int layout, float sign, void* stream) {
    if (tokens < 0 || tokens > kMostTokens || heads < 1 || heads > (1 << 20) || dim < 8 || dim > 512) return NF4_EINVAL;
    if (dim % 8) return NF4_ESHAPE;
    if (is_bf16 != 0 && is_bf16 != 1) return NF4_EUNSUPPORTED;
    if (tokens == 0) return NF4_OK;
    if (bad(x) || bad(y)) return NF4_EINVAL;
    const int step = is_bf16 ? 8 : 4;
    for (int64_t s : {xt, xh, yt, yh})
        if (s % step) return NF4_ESHAPE;
    if (xh < dim || yh < dim || xt < 0) return NF4_EINVAL;
    // the output's heads lie apart: all of a token's before the next token's, or
    // all of a head's tokens before the next head's (quotients: no sum overflows)
    auto within = [&](int64_t n, int64_t step, int64_t next) { return step >= dim && next >= dim && (next - dim) / step >= n - 1; };
    if (!within(heads, yh, yt) && !within(tokens, yt, yh)) return NF4_EINVAL;
    if (x == y && (xt != yt || xh != yh)) return NF4_EINVAL;
    kv::Rope r;
    if (const int rc = rope_of(positions, table, max_pos, rot, layout, dim, false, &r)) return rc;
    return kv::rope(x, xt, xh, y, yt, yh, tokens, heads, dim, is_bf16 == 1, r, sign,
                    static_cast<hipStream_t>(stream));
}

}  // namespace

namespace kv {

int launch_status() {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return NF4_OK;
    g_last_hip_error = int(e);
    return NF4_ELAUNCH;
}

}  // namespace kv

extern "C" {

int nf4_kv_last_hip_error(void) { return g_last_hip_error; }

int nf4_rope_table(float* table, int64_t max_pos, int32_t rot, float base, const nf4_rope_scaling* scaling,
                   void* stream) {
    if (bad(table) || !scaling || max_pos < 1) return NF4_EINVAL;
    if (rot < 2 || rot > 512 || rot % 2) return NF4_ESHAPE;
    if (max_pos > (int64_t(1) << 32) / rot - 256) return NF4_EINVAL;  // a thread for each pair, 2^31 of them
    if (!isfinite(base) || base <= 1.0f || !isfinite(scaling->amplitude)) return NF4_EINVAL;
    const nf4_rope_scaling& s = *scaling;
    if (s.kind < NF4_ROPE_NONE || s.kind > NF4_ROPE_PARTS) return NF4_EUNSUPPORTED;
    if (s.kind != NF4_ROPE_NONE && !(isfinite(s.factor) && s.factor > 0.0f)) return NF4_EINVAL;
    if (s.kind == NF4_ROPE_BASE && rot == 2) return NF4_ESHAPE;
    if (s.kind == NF4_ROPE_PARTS && !(isfinite(s.high) && s.low >= 0.0f && s.low < s.high && isfinite(s.original) &&
                                      s.original > 0.0f))
        return NF4_EINVAL;
    return kv::rope_table(table, max_pos, rot, base, s, static_cast<hipStream_t>(stream));
}

int nf4_rope_forward(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* y, int64_t y_token_stride,
                     int64_t y_head_stride, int64_t tokens, int32_t n_heads, int32_t head_dim, int32_t is_bf16,
                     const int32_t* positions, const float* table, int64_t max_pos, int32_t rot, int32_t layout,
                     void* stream) {
    return rope_call(x, x_token_stride, x_head_stride, y, y_token_stride, y_head_stride, tokens, n_heads, head_dim,
                     is_bf16, positions, table, max_pos, rot, layout, 1.0f, stream);
}

int nf4_rope_backward(const void* dy, int64_t dy_token_stride, int64_t dy_head_stride, void* dx,
                      int64_t dx_token_stride, int64_t dx_head_stride, int64_t tokens, int32_t n_heads,
                      int32_t head_dim, int32_t is_bf16, const int32_t* positions, const float* table,
                      int64_t max_pos, int32_t rot, int32_t layout, void* stream) {
    return rope_call(dy, dy_token_stride, dy_head_stride, dx, dx_token_stride, dx_head_stride, tokens, n_heads,
                     head_dim, is_bf16, positions, table, max_pos, rot, layout, -1.0f, stream);
}

int nf4_kv_plan(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* done, int32_t batch,
                int32_t* block_table, int32_t table_width, int32_t page_size, int32_t* free_pages, int32_t capacity,
                const int32_t* free_state, int32_t max_tokens, int32_t* kv_lens_out, int32_t* cu_new, int64_t* slots,
                int32_t* positions, int32_t* free_out, int32_t* refused, void* stream) {
    if (batch < 1 || table_width < 1 || capacity < 1 || max_tokens < 0) return NF4_EINVAL;
    if (batch > 4096) return NF4_EUNSUPPORTED;
    if (capacity > (1 << 30) || max_tokens > (1 << 30)) return NF4_EINVAL;
    const int shift = page_shift(page_size);
    if (shift < 0) return NF4_EUNSUPPORTED;
    const void* const words[] = {kv_lens, new_lens, block_table, free_pages, free_state, kv_lens_out, cu_new, free_out,
                                 refused};
    for (const void* p : words)
        if (!p || (reinterpret_cast<uintptr_t>(p) & 3)) return NF4_EINVAL;
    if (reinterpret_cast<uintptr_t>(done) & 3) return NF4_EINVAL;
    if (max_tokens > 0 && (!slots || (reinterpret_cast<uintptr_t>(slots) & 7) || !positions ||
                           (reinterpret_cast<uintptr_t>(positions) & 3)))
        return NF4_EINVAL;
    if (kv_lens_out == kv_lens || kv_lens_out == new_lens || cu_new == kv_lens || cu_new == new_lens ||
        free_out == free_state)
        return NF4_EINVAL;
    return kv::plan(kv_lens, new_lens, done, batch, block_table, table_width, shift, free_pages, capacity, free_state,
                    max_tokens, kv_lens_out, cu_new, slots, positions, free_out, refused,
                    static_cast<hipStream_t>(stream));
}

int nf4_kv_append(const nf4_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                  int64_t v_stride, const int64_t* slots, int64_t tokens, const uint16_t* q, int64_t q_stride,
                  uint16_t* q_out, int64_t q_out_stride, int32_t q_heads, const int32_t* positions,
                  const float* table, int64_t max_pos, int32_t rot, int32_t layout, void* stream) {
    kv::Cache c;
    if (const int rc = cache_of(cache, &c)) return rc;
    if (tokens < 0 || tokens > kMostTokens) return NF4_EINVAL;
    if (tokens == 0) return NF4_OK;
    kv::Rope r;
    if (const int rc = rope_of(positions, table, max_pos, rot, layout, c.head_dim, true, &r)) return rc;
    if (bad(k) || bad(v) || !slots || (reinterpret_cast<uintptr_t>(slots) & 7)) return NF4_EINVAL;
    const int64_t row = int64_t(c.n_heads) * c.head_dim;
    if (k_stride % 8 || v_stride % 8) return NF4_ESHAPE;
    if (k_stride < row || v_stride < row) return NF4_EINVAL;
    if (q) {
        if (rot == 0 || bad(q) || bad(q_out) || q == q_out || q_heads < 1 || q_heads > (1 << 20)) return NF4_EINVAL;
        if (q_stride % 8 || q_out_stride % 8) return NF4_ESHAPE;
        const int64_t qrow = int64_t(q_heads) * c.head_dim;
        if (q_stride < qrow || q_out_stride < qrow) return NF4_EINVAL;
    }
    return kv::append(c, k, k_stride, v, v_stride, slots, tokens, q, q_stride, q_out, q_out_stride, q_heads, r,
                      static_cast<hipStream_t>(stream));
}

int nf4_kv_read(const nf4_kv_cache* cache, const int64_t* slots, int64_t tokens, uint16_t* k_out, uint16_t* v_out,
                void* stream) {
    kv::Cache c;
    if (const int rc = cache_of(cache, &c)) return rc;
    if (tokens < 0 || tokens > kMostTokens) return NF4_EINVAL;
    if (tokens == 0 || (!k_out && !v_out)) return NF4_OK;
    if (!slots || (reinterpret_cast<uintptr_t>(slots) & 7)) return NF4_EINVAL;
    if ((k_out && bad(k_out)) || (v_out && bad(v_out))) return NF4_EINVAL;
    return kv::read(c, slots, tokens, k_out, v_out, static_cast<hipStream_t>(stream));
}

namespace {

// The shape checks shared by the call and its workspace query.
int attn_shape(int batch, int q_heads, int n_heads, int max_q, int max_len, int window, int sinks) {
    if (batch < 1 || batch > 65535 || max_q < 0 || max_len < 0 || window < 0 || sinks < 0) return NF4_EINVAL;
    if (q_heads < 1 || n_heads < 1 || n_heads > 1024) return NF4_EINVAL;
    if (q_heads % n_heads || q_heads / n_heads > 128) return NF4_ESHAPE;
    if (int64_t(max_q) * (q_heads / n_heads) > 0x7fffffff - 4096) return NF4_EINVAL;
    if (max_len > 0x7fffffff - 4096) return NF4_EINVAL;
    return NF4_OK;
}

int attn(bool zero_rest, const nf4_kv_cache* cache, const uint16_t* q, int64_t q_stride, int64_t total_q, int32_t q_heads,
         const int32_t* cu_q, const int32_t* kv_lens, const int32_t* block_table, int32_t table_width, int32_t batch,
         int32_t max_q, int32_t max_len, float scale, int32_t window, int32_t sinks, uint16_t* out, int64_t out_stride,
         void* ws, size_t ws_bytes, void* stream) {
    kv::Cache c;
    if (const int rc = cache_of(cache, &c)) return rc;
    if (const int rc = attn_shape(batch, q_heads, c.n_heads, max_q, max_len, window, sinks)) return rc;
    if (total_q < 0 || total_q > 0x7fffffff || !isfinite(scale)) return NF4_EINVAL;
    if (table_width < 0 || max_len > int64_t(table_width) << c.pshift) return NF4_EINVAL;
    if (total_q == 0 || (max_q == 0 && !zero_rest)) return NF4_OK;
    if (bad(q) || bad(out) || q == out) return NF4_EINVAL;
    const int32_t* const words[] = {cu_q, kv_lens};
    for (const int32_t* p : words)
        if (!p || (reinterpret_cast<uintptr_t>(p) & 3)) return NF4_EINVAL;
    if (max_len > 0 && (!block_table || (reinterpret_cast<uintptr_t>(block_table) & 3))) return NF4_EINVAL;
    if (q_stride % 8 || out_stride % 8) return NF4_ESHAPE;
    const int64_t row = int64_t(q_heads) * c.head_dim;
    if (q_stride < row || out_stride < row) return NF4_EINVAL;
    const kv::Attn a = {q, q_stride, total_q, out, out_stride, cu_q, kv_lens, block_table, table_width, batch,
                        q_heads, max_q, max_len, window, sinks, scale};
    const size_t need = kv::attention_ws_bytes(c, a);
    if (need && (bad(ws) || ws_bytes < need)) return NF4_EWORKSPACE;
    return kv::attention(c, a, zero_rest, ws, static_cast<hipStream_t>(stream));
}

}  // namespace

size_t nf4_kv_attention_ws_bytes(int32_t batch, int32_t q_heads, int32_t n_heads, int32_t head_dim, int32_t max_q,
                                 int32_t max_len, int32_t window, int32_t sinks) {
    if (attn_shape(batch, q_heads, n_heads, max_q, max_len, window, sinks)) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    kv::Cache c = {};
    c.n_heads = n_heads;
    c.head_dim = head_dim;
    kv::Attn a = {};
    a.batch = batch, a.q_heads = q_heads, a.max_q = max_q, a.max_len = max_len, a.window = window, a.sinks = sinks;
    return kv::attention_ws_bytes(c, a);
}

int nf4_kv_attention(const nf4_kv_cache* cache, const uint16_t* q, int64_t q_stride, int64_t total_q,
                     int32_t q_heads, const int32_t* cu_q, const int32_t* kv_lens, const int32_t* block_table,
                     int32_t table_width, int32_t batch, int32_t max_q, int32_t max_len, float scale, int32_t window,
                     int32_t sinks, uint16_t* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
    return attn(false, cache, q, q_stride, total_q, q_heads, cu_q, kv_lens, block_table, table_width, batch, max_q,
                max_len, scale, window, sinks, out, out_stride, ws, ws_bytes, stream);
}

int nf4_kv_attention_padded(const nf4_kv_cache* cache, const uint16_t* q, int64_t q_stride, int64_t total_q,
                            int32_t q_heads, const int32_t* cu_q, const int32_t* kv_lens, const int32_t* block_table,
                            int32_t table_width, int32_t batch, int32_t max_q, int32_t max_len, float scale,
                            int32_t window, int32_t sinks, uint16_t* out, int64_t out_stride, void* ws,
                            size_t ws_bytes, void* stream) {
    return attn(true, cache, q, q_stride, total_q, q_heads, cu_q, kv_lens, block_table, table_width, batch, max_q,
                max_len, scale, window, sinks, out, out_stride, ws, ws_bytes, stream);
}

}  // extern "C"
