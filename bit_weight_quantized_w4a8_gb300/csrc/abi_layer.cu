// abi_layer.cu -- the extern "C" entry points of the decoder layer around the
// linears (include/w4a8.h): argument checks on the host, launches on the
// caller's stream; nothing allocates or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/w4a8.h"
#include "abi_status.h"
#include "kernels.h"

namespace {

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return w4a8::status_fail(code, buf);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_type(int t) { return t == W4A8_T_F32 || t == W4A8_T_F16; }
int size_of(int t) { return t == W4A8_T_F16 ? 2 : 4; }

int check_flags(const char* who, unsigned flags) {
    if (flags & ~W4A8_LAUNCH_PDL) return fail(W4A8_ERR_SHAPE, "%s: unknown flags 0x%x", who, flags);
    return W4A8_OK;
}

int check_cache(const char* who, const kvq_cache_t* c) {
    if (!c || !c->k || !c->v || !c->ks || !c->vs) return fail(W4A8_ERR_NULL, "%s: NULL pointer in the cache", who);
    if (c->pages < 1 || c->pages > 0x7FFFFFFF)
        return fail(W4A8_ERR_SHAPE, "%s: pages=%lld outside [1, 2^31-1]", who, (long long)c->pages);
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)))
        return fail(W4A8_ERR_SHAPE, "%s: page=%d must be 16, 32, 64, 128 or 256", who, c->page);
    if (c->heads < 1 || c->heads > 1024) return fail(W4A8_ERR_SHAPE, "%s: heads=%d outside [1, 1024]", who, c->heads);
    if (c->dim != 64 && c->dim != 128 && c->dim != 256)
        return fail(W4A8_ERR_SHAPE, "%s: dim=%d must be 64, 128 or 256", who, c->dim);
    if (c->bits != 8 && c->bits != 4) return fail(W4A8_ERR_SHAPE, "%s: bits=%d must be 8 or 4", who, c->bits);
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->ks, 4) || !aligned(c->vs, 4))
        return fail(W4A8_ERR_ALIGN, "%s: the cache's codes need 16-byte, its scales 4-byte alignment", who);
    return W4A8_OK;
}

int check_batch(const char* who, const kvq_batch_t* b) {
    if (!b || !b->cu || !b->start || !b->table) return fail(W4A8_ERR_NULL, "%s: NULL pointer in the batch", who);
    if (b->seqs < 1 || b->seqs > 65536 || b->tokens < 1 || b->tokens > 0x7FFFFFFF || b->max_pages < 1 ||
        b->max_pages > 0x7FFFFFFF)
        return fail(W4A8_ERR_SHAPE, "%s: seqs=%lld, tokens=%lld or max_pages=%lld out of range", who,
                    (long long)b->seqs, (long long)b->tokens, (long long)b->max_pages);
    if (!aligned(b->cu, 4) || !aligned(b->start, 4) || !aligned(b->table, 4))
        return fail(W4A8_ERR_ALIGN, "%s: the batch's arrays need 4-byte alignment", who);
    return W4A8_OK;
}

int check_rope(const char* who, const int32_t* pos, const double* freqs, int rot, int dim, float mscale) {
    if (!pos || !freqs) return fail(W4A8_ERR_NULL, "%s: NULL positions or frequencies", who);
    if (rot < 8 || rot > dim || rot % 8)
        return fail(W4A8_ERR_SHAPE, "%s: rot=%d must be a multiple of 8 in [8, %d]", who, rot, dim);
    if (!std::isfinite(mscale)) return fail(W4A8_ERR_SHAPE, "%s: mscale is not finite", who);
    if (!aligned(pos, 4) || !aligned(freqs, 8))
        return fail(W4A8_ERR_ALIGN, "%s: positions need 4-byte, frequencies 8-byte alignment", who);
    return W4A8_OK;
}

// Axis of each pair: a host array of rot / 2 entries.
int check_axis(const char* who, int axes, const uint8_t* axis, int rot) {
    if (!axis) return fail(W4A8_ERR_NULL, "%s: NULL axis", who);
    if (axes < 1 || axes > ROPE_MAX_AXES)
        return fail(W4A8_ERR_SHAPE, "%s: axes=%d outside [1, %d]", who, axes, ROPE_MAX_AXES);
    for (int i = 0; i < rot / 2; ++i)
        if (axis[i] >= axes)
            return fail(W4A8_ERR_SHAPE, "%s: pair %d is on axis %d of %d", who, i, (int)axis[i], axes);
    return W4A8_OK;
}

// Rows of `heads` vectors of dim values, ld elements apart.
int check_rows(const char* who, const char* name, const void* p, int type, int64_t ld, int64_t heads, int dim) {
    if (!p) return fail(W4A8_ERR_NULL, "%s: NULL %s", who, name);
    if (ld < heads * dim || ld % 4)
        return fail(W4A8_ERR_SHAPE, "%s: rows of %s are %lld elements apart (at least %lld, a multiple of 4)", who,
                    name, (long long)ld, (long long)(heads * dim));
    if (!aligned(p, type == W4A8_T_F16 ? 8 : 16))
        return fail(W4A8_ERR_ALIGN, "%s: %s needs 16-byte (binary16: 8-byte) alignment", who, name);
    return W4A8_OK;
}

}  // namespace

extern "C" {

int add_norm(const void* r, int r_type, const void* y, int y_type, const float* post_w, const float* gate,
             int64_t ld_gate, const float* w, int64_t M, int64_t N, float alpha, float beta, float eps, void* r_out,
             uint16_t* X, int8_t* Xq, float* sa, unsigned flags, void* stream) {
    if (!r || (!Xq) != (!sa) || (!r_out && !X && !Xq) || ((X || Xq) && !w))
        return fail(W4A8_ERR_NULL, "add_norm: NULL pointer");
    if (!is_type(r_type) || (y && !is_type(y_type))) return fail(W4A8_ERR_SHAPE, "add_norm: unknown type");
    if (M < 1 || M > 0x7FFFFFFF || N < 1 || N > W4A8_NORM_MAX_N)
        return fail(W4A8_ERR_SHAPE, "add_norm: M=%lld or N=%lld out of range", (long long)M, (long long)N);
    if (gate && ld_gate != 0 && ld_gate < N)
        return fail(W4A8_ERR_SHAPE, "add_norm: ld_gate=%lld must be 0 or at least N", (long long)ld_gate);
    if (!std::isfinite(alpha) || !std::isfinite(beta) || !std::isfinite(eps) || eps < 0.f)
        return fail(W4A8_ERR_SHAPE, "add_norm: alpha, beta and eps must be finite, eps >= 0");
    if (Xq && N % 8) return fail(W4A8_ERR_SHAPE, "add_norm: codes need N %% 8 == 0, got %lld", (long long)N);
    int st = check_flags("add_norm", flags);
    if (st != W4A8_OK) return st;
    if (!aligned(r, size_of(r_type)) || !aligned(r_out, size_of(r_type)) || (y && !aligned(y, size_of(y_type))) ||
        !aligned(post_w, 4) || !aligned(gate, 4) || !aligned(w, 4) || !aligned(X, 2) || !aligned(sa, 4))
        return fail(W4A8_ERR_ALIGN, "add_norm: a tensor is not aligned to its element");
    const bool vec = N % 8 == 0 && aligned(r, 16) && aligned(r_out, 16) && aligned(y, 16) && aligned(post_w, 16) &&
                     (!gate || (aligned(gate, 16) && ld_gate % 4 == 0)) && aligned(w, 16) && aligned(X, 16) &&
                     aligned(Xq, 8);
    return w4a8::status_done(w4a8::launch_add_norm(r, r_type, y, y_type, post_w, gate, ld_gate, w, M, (int)N, alpha,
                                                   beta, eps, r_out, X, Xq, sa, vec, flags,
                                                   static_cast<cudaStream_t>(stream)),
                             "add_norm launch");
}

int rope_frequencies(int rot, double base, int scaling, double factor, double old_ctx, double low, double high,
                     double* freqs, float* mscale) {
    if (!freqs) return fail(W4A8_ERR_NULL, "rope_frequencies: NULL pointer");
    if (rot < 8 || rot > 256 || rot % 8)
        return fail(W4A8_ERR_SHAPE, "rope_frequencies: rot=%d must be a multiple of 8 in [8, 256]", rot);
    if (scaling < ROPE_PLAIN || scaling > ROPE_BANDS)
        return fail(W4A8_ERR_SHAPE, "rope_frequencies: unknown scaling %d", scaling);
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor))
        return fail(W4A8_ERR_SHAPE, "rope_frequencies: needs base > 1 and factor >= 1");
    const bool parts = scaling == ROPE_YARN || scaling == ROPE_BANDS;
    if (parts && (!(old_ctx >= 1.0) || !std::isfinite(old_ctx) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
        return fail(W4A8_ERR_SHAPE, "rope_frequencies: needs old_ctx >= 1 and 0 < low < high");
    const double pi = 3.14159265358979323846;
    if (scaling == ROPE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
    // the pair index at which a pair turns n times within old_ctx positions
    auto pair_of = [&](double n) { return rot * std::log(old_ctx / (n * 2.0 * pi)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == ROPE_YARN) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), (double)(rot - 1));
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double g = f;
        if (scaling == ROPE_LINEAR) {
            g = f / factor;
        } else if (scaling == ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - first) / (last - first), 0.0), 1.0);
            g = f / factor * ramp + f * (1.0 - ramp);
        } else if (scaling == ROPE_BANDS) {
            const double turns = old_ctx * f / (2.0 * pi);  // old_ctx / wavelength
            const double keep = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
            g = f / factor * (1.0 - keep) + f * keep;
        }
        freqs[i] = g;
    }
    if (mscale) *mscale = scaling == ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return w4a8::status_done(cudaSuccess, "");
}

// axes 0: one axis, no map.
static int rotate_rows(const char* who, const void* X, int x_type, int64_t ld_x, int64_t tokens, int heads, int dim,
                       const int32_t* pos, int axes, const uint8_t* axis, const double* freqs, int rot, int interleaved,
                       float mscale, void* Y, int y_type, int64_t ld_y, unsigned flags, void* stream) {
    if (!is_type(x_type) || !is_type(y_type)) return fail(W4A8_ERR_SHAPE, "%s: unknown type", who);
    if (dim != 64 && dim != 128 && dim != 256)
        return fail(W4A8_ERR_SHAPE, "%s: dim=%d must be 64, 128 or 256", who, dim);
    if (tokens < 1 || tokens > 0x7FFFFFFF || heads < 1 || heads > 16384)
        return fail(W4A8_ERR_SHAPE, "%s: tokens=%lld or heads=%d out of range", who, (long long)tokens, heads);
    int st;
    if ((st = check_rows(who, "X", X, x_type, ld_x, heads, dim)) != W4A8_OK) return st;
    if ((st = check_rows(who, "Y", Y, y_type, ld_y, heads, dim)) != W4A8_OK) return st;
    if (X == Y && (x_type != y_type || ld_x != ld_y))
        return fail(W4A8_ERR_SHAPE, "%s: in place needs one type and one row distance", who);
    if ((st = check_rope(who, pos, freqs, rot, dim, mscale)) != W4A8_OK) return st;
    if (axes != 0 && (st = check_axis(who, axes, axis, rot)) != W4A8_OK) return st;
    if ((st = check_flags(who, flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    return w4a8::status_done(w4a8::launch_rope_rotate(X, x_type, ld_x, tokens, heads, dim, pos, axis, freqs, rot,
                                                      interleaved != 0, mscale, Y, y_type, ld_y, sms, flags,
                                                      static_cast<cudaStream_t>(stream)),
                             who);
}

int rope_rotate(const void* X, int x_type, int64_t ld_x, int64_t tokens, int heads, int dim, const int32_t* pos,
                const double* freqs, int rot, int interleaved, float mscale, void* Y, int y_type, int64_t ld_y,
                unsigned flags, void* stream) {
    return rotate_rows("rope_rotate", X, x_type, ld_x, tokens, heads, dim, pos, 0, nullptr, freqs, rot, interleaved, mscale,
                  Y, y_type, ld_y, flags, stream);
}

int rope_rotate_axes(const void* X, int x_type, int64_t ld_x, int64_t tokens, int heads, int dim, const int32_t* pos,
                     int axes, const uint8_t* axis, const double* freqs, int rot, int interleaved, float mscale,
                     void* Y, int y_type, int64_t ld_y, unsigned flags, void* stream) {
    if (axes == 0) return fail(W4A8_ERR_SHAPE, "rope_rotate_axes: axes=0 outside [1, %d]", ROPE_MAX_AXES);
    return rotate_rows("rope_rotate_axes", X, x_type, ld_x, tokens, heads, dim, pos, axes, axis, freqs, rot, interleaved,
                  mscale, Y, y_type, ld_y, flags, stream);
}

static int write_tokens(const char* who, const kvq_cache_t* cache, const kvq_batch_t* batch, const void* K, int64_t ld_k,
                        const void* V, int64_t ld_v, const void* Q, int64_t ld_q, int heads_q, int x_type, const int32_t* pos,
                        int axes, const uint8_t* axis, const double* freqs, int rot, int interleaved, float mscale,
                        uint16_t* Q_out, unsigned flags, void* stream) {
    int st;
    if ((st = check_cache(who, cache)) != W4A8_OK) return st;
    if ((st = check_batch(who, batch)) != W4A8_OK) return st;
    if (!is_type(x_type)) return fail(W4A8_ERR_SHAPE, "%s: unknown type", who);
    if ((st = check_rows(who, "K", K, x_type, ld_k, cache->heads, cache->dim)) != W4A8_OK) return st;
    if ((st = check_rows(who, "V", V, x_type, ld_v, cache->heads, cache->dim)) != W4A8_OK) return st;
    if ((!Q) != (!Q_out)) return fail(W4A8_ERR_NULL, "%s: Q and Q_out come together", who);
    if (Q) {
        if (heads_q < 1 || heads_q > 16384)
            return fail(W4A8_ERR_SHAPE, "%s: heads_q=%d outside [1, 16384]", who, heads_q);
        if ((st = check_rows(who, "Q", Q, x_type, ld_q, heads_q, cache->dim)) != W4A8_OK) return st;
        if (!aligned(Q_out, 8)) return fail(W4A8_ERR_ALIGN, "%s: Q_out needs 8-byte alignment", who);
    }
    if (freqs && (st = check_rope(who, pos, freqs, rot, cache->dim, mscale)) != W4A8_OK) return st;
    if (axes != 0 && (st = check_axis(who, axes, axis, rot)) != W4A8_OK) return st;
    if ((st = check_flags(who, flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    return w4a8::status_done(w4a8::launch_kvq_write(*cache, *batch, K, ld_k, V, ld_v, Q, ld_q, heads_q, x_type, pos,
                                                    axis, freqs, rot, interleaved != 0, mscale, Q_out, sms, flags,
                                                    static_cast<cudaStream_t>(stream)),
                             who);
}

int kvq_write(const kvq_cache_t* cache, const kvq_batch_t* batch, const void* K, int64_t ld_k, const void* V,
              int64_t ld_v, const void* Q, int64_t ld_q, int heads_q, int x_type, const int32_t* pos,
              const double* freqs, int rot, int interleaved, float mscale, uint16_t* Q_out, unsigned flags,
              void* stream) {
    return write_tokens("kvq_write", cache, batch, K, ld_k, V, ld_v, Q, ld_q, heads_q, x_type, pos, 0, nullptr, freqs, rot,
                 interleaved, mscale, Q_out, flags, stream);
}

int kvq_write_axes(const kvq_cache_t* cache, const kvq_batch_t* batch, const void* K, int64_t ld_k, const void* V,
                   int64_t ld_v, const void* Q, int64_t ld_q, int heads_q, int x_type, const int32_t* pos, int axes,
                   const uint8_t* axis, const double* freqs, int rot, int interleaved, float mscale, uint16_t* Q_out,
                   unsigned flags, void* stream) {
    if (axes == 0) return fail(W4A8_ERR_SHAPE, "kvq_write_axes: axes=0 outside [1, %d]", ROPE_MAX_AXES);
    if (!freqs) return fail(W4A8_ERR_NULL, "kvq_write_axes: NULL positions or frequencies");
    return write_tokens("kvq_write_axes", cache, batch, K, ld_k, V, ld_v, Q, ld_q, heads_q, x_type, pos, axes, axis, freqs, rot,
                 interleaved, mscale, Q_out, flags, stream);
}

int kvq_read(const kvq_cache_t* cache, const kvq_batch_t* batch, void* K, void* V, int y_type, unsigned flags,
             void* stream) {
    int st;
    if ((st = check_cache("kvq_read", cache)) != W4A8_OK) return st;
    if ((st = check_batch("kvq_read", batch)) != W4A8_OK) return st;
    if (!K || !V) return fail(W4A8_ERR_NULL, "kvq_read: NULL output");
    if (!is_type(y_type)) return fail(W4A8_ERR_SHAPE, "kvq_read: unknown type");
    if (!aligned(K, 16) || !aligned(V, 16)) return fail(W4A8_ERR_ALIGN, "kvq_read: K and V need 16-byte alignment");
    if ((st = check_flags("kvq_read", flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    return w4a8::status_done(
        w4a8::launch_kvq_read(*cache, *batch, K, V, y_type, sms, flags, static_cast<cudaStream_t>(stream)),
        "kvq_read launch");
}

int kvq_keep(const kvq_cache_t* cache, const kvq_batch_t* batch, const int32_t* keep, unsigned flags, void* stream) {
    int st;
    if ((st = check_cache("kvq_keep", cache)) != W4A8_OK) return st;
    if ((st = check_batch("kvq_keep", batch)) != W4A8_OK) return st;
    if (!keep) return fail(W4A8_ERR_NULL, "kvq_keep: NULL keep");
    if (!aligned(keep, 4)) return fail(W4A8_ERR_ALIGN, "kvq_keep: keep needs 4-byte alignment");
    if ((st = check_flags("kvq_keep", flags)) != W4A8_OK) return st;
    return w4a8::status_done(
        w4a8::launch_kvq_keep(*cache, *batch, keep, flags, static_cast<cudaStream_t>(stream)), "kvq_keep launch");
}

static int check_attention(const kvq_cache_t* cache, const kvq_batch_t* batch, int heads_q) {
    int st;
    if ((st = check_cache("kvq_attention", cache)) != W4A8_OK) return st;
    if ((st = check_batch("kvq_attention", batch)) != W4A8_OK) return st;
    if (heads_q < cache->heads || heads_q % cache->heads || heads_q > 1024 * cache->heads)
        return fail(W4A8_ERR_SHAPE, "kvq_attention: heads_q=%d must be 1 to 1024 times heads=%d", heads_q,
                    cache->heads);
    if (batch->tokens * heads_q > 0x7FFFFFFF)
        return fail(W4A8_ERR_SHAPE, "kvq_attention: tokens * heads_q = %lld above 2^31-1",
                    (long long)(batch->tokens * heads_q));
    return W4A8_OK;
}

size_t kvq_attention_workspace_bytes(const kvq_cache_t* cache, const kvq_batch_t* batch, int heads_q) {
    int sms = 0;
    if (check_attention(cache, batch, heads_q) != W4A8_OK || w4a8::status_sm_count(&sms) != W4A8_OK) return 0;
    return w4a8::kvq_attn_workspace(*cache, *batch, heads_q, sms);
}

int kvq_attention(const kvq_cache_t* cache, const kvq_batch_t* batch, const uint16_t* Q, int heads_q,
                  const uint64_t* mask, float scale, uint16_t* out, void* ws, size_t ws_bytes, unsigned flags,
                  void* stream) {
    int st;
    if ((st = check_attention(cache, batch, heads_q)) != W4A8_OK) return st;
    if (!Q || !out) return fail(W4A8_ERR_NULL, "kvq_attention: NULL pointer");
    if (!std::isfinite(scale)) return fail(W4A8_ERR_SHAPE, "kvq_attention: scale is not finite");
    if (!aligned(Q, 16) || !aligned(out, 16) || !aligned(mask, 8))
        return fail(W4A8_ERR_ALIGN, "kvq_attention: Q and out need 16-byte, mask 8-byte alignment");
    if ((st = check_flags("kvq_attention", flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    const size_t need = w4a8::kvq_attn_workspace(*cache, *batch, heads_q, sms);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(W4A8_ERR_WORKSPACE, "kvq_attention: workspace of %zu bytes needed, got %zu", need,
                    ws ? ws_bytes : (size_t)0);
    if (need > 0 && !aligned(ws, 256)) return fail(W4A8_ERR_ALIGN, "kvq_attention: workspace needs 256-byte alignment");
    return w4a8::status_done(w4a8::launch_kvq_attention(*cache, *batch, Q, heads_q, mask, scale, out, ws, sms, flags,
                                                        static_cast<cudaStream_t>(stream)),
                             "kvq_attention launch");
}

}  // extern "C"
