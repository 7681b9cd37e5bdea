// abi_step.cu -- the extern "C" entry points of a serving step around the
// layers and of the linear with e4m3 blocks (include/w4a8.h): argument checks on the
// host, launches on the caller's stream; nothing allocates or synchronises.
#include <cuda_runtime.h>

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
constexpr int64_t kIntMax = 0x7FFFFFFF;

int check_flags(const char* who, unsigned flags) {
    if (flags & ~W4A8_LAUNCH_PDL) return fail(W4A8_ERR_SHAPE, "%s: unknown flags 0x%x", who, flags);
    return W4A8_OK;
}

int check_workspace(const char* who, const void* ws, size_t have, size_t need) {
    if (need == 0) return W4A8_OK;
    if (!ws || have < need)
        return fail(W4A8_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, got %zu", who, need, ws ? have : (size_t)0);
    if (!aligned(ws, 256)) return fail(W4A8_ERR_ALIGN, "%s: workspace needs 256-byte alignment", who);
    return W4A8_OK;
}

int check_pool(const char* who, const kvq_pool_t* p) {
    if (!p || !p->table || !p->held || !p->stack || !p->top) return fail(W4A8_ERR_NULL, "%s: NULL pointer in the pool", who);
    if (p->seqs < 1 || p->seqs > 65536 || p->max_pages < 1 || p->max_pages > kIntMax || p->pages < 1 || p->pages > kIntMax)
        return fail(W4A8_ERR_SHAPE, "%s: seqs=%lld, max_pages=%lld or pages=%lld out of range", who, (long long)p->seqs,
                    (long long)p->max_pages, (long long)p->pages);
    if (p->page < 16 || p->page > 256 || (p->page & (p->page - 1)))
        return fail(W4A8_ERR_SHAPE, "%s: page=%d must be 16, 32, 64, 128 or 256", who, p->page);
    if (!aligned(p->table, 4) || !aligned(p->held, 4) || !aligned(p->stack, 4) || !aligned(p->top, 4))
        return fail(W4A8_ERR_ALIGN, "%s: the pool's arrays need 4-byte alignment", who);
    return W4A8_OK;
}

int check_linear(const char* who, int64_t M, int64_t K, int64_t N) {
    if (M < 1 || M > 1 << 24) return fail(W4A8_ERR_SHAPE, "%s: M=%lld outside [1, 2^24]", who, (long long)M);
    if (K < 16 || K > 131072 || K % 16)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a multiple of 16 in [16, 131072]", who, (long long)K);
    if (N < 1 || N > kIntMax) return fail(W4A8_ERR_SHAPE, "%s: N=%lld outside [1, 2^31-1]", who, (long long)N);
    if (M * N > (int64_t)1 << 43) return fail(W4A8_ERR_SHAPE, "%s: M * N above 2^43", who);
    return W4A8_OK;
}

int check_vocab(const char* who, int64_t tokens, int64_t vocab) {
    if (tokens < 1 || tokens > kIntMax || vocab < 1 || vocab > 1 << 22)
        return fail(W4A8_ERR_SHAPE, "%s: tokens=%lld or vocab=%lld out of range", who, (long long)tokens, (long long)vocab);
    return W4A8_OK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int64_t blocks(int64_t k) { return (k + F8_BLOCK - 1) / F8_BLOCK; }
// f8_linear's workspace: codes, scales.
size_t linear_scales_at(int64_t M, int64_t K) { return round256((size_t)M * K); }
size_t linear_bytes(int64_t M, int64_t K) { return linear_scales_at(M, K) + round256((size_t)M * blocks(K) * 4); }

cudaStream_t st_of(void* stream) { return static_cast<cudaStream_t>(stream); }

}  // namespace

extern "C" {

size_t kvq_plan_workspace_bytes(const kvq_pool_t* pool) {
    return check_pool("kvq_plan", pool) == W4A8_OK ? w4a8::kvq_plan_workspace(*pool) : 0;
}

int kvq_plan(const kvq_pool_t* pool, int32_t* lens, const int32_t* grow, const int32_t* add, const uint64_t* mask,
             int64_t tokens, int32_t* cu, int32_t* pos, int64_t* slot, int32_t* seq, void* ws, size_t ws_bytes,
             unsigned flags, void* stream) {
    int st;
    if ((st = check_pool("kvq_plan", pool)) != W4A8_OK) return st;
    if (!lens || !add || !cu) return fail(W4A8_ERR_NULL, "kvq_plan: NULL pointer");
    if (tokens < 1 || tokens > kIntMax) return fail(W4A8_ERR_SHAPE, "kvq_plan: tokens=%lld out of range", (long long)tokens);
    if (!aligned(lens, 4) || !aligned(grow, 4) || !aligned(add, 4) || !aligned(cu, 4) || !aligned(pos, 4) ||
        !aligned(seq, 4) || !aligned(mask, 8) || !aligned(slot, 8))
        return fail(W4A8_ERR_ALIGN, "kvq_plan: mask and slot need 8-byte, the other arrays 4-byte alignment");
    if ((st = check_flags("kvq_plan", flags)) != W4A8_OK) return st;
    if ((st = check_workspace("kvq_plan", ws, ws_bytes, w4a8::kvq_plan_workspace(*pool))) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    return w4a8::status_done(
        w4a8::launch_kvq_plan(*pool, lens, grow, add, mask, tokens, cu, pos, slot, seq, ws, sms, flags, st_of(stream)),
        "kvq_plan launch");
}

size_t draft_verify_workspace_bytes(int64_t tokens, int64_t vocab) {
    int sms = 0;
    if (check_vocab("draft_verify", tokens, vocab) != W4A8_OK || w4a8::status_sm_count(&sms) != W4A8_OK) return 0;
    return w4a8::draft_verify_workspace(tokens, vocab, sms);
}

int draft_verify(const void* L, int l_type, int64_t ld_l, int64_t vocab, const int32_t* cu, int64_t seqs,
                 int64_t tokens, const int32_t* ids, const uint64_t* mask, const void* Q, int q_type, int64_t ld_q,
                 const float* temp, const float* u, int32_t* keep, int32_t* out, int32_t* count, void* ws,
                 size_t ws_bytes, unsigned flags, void* stream) {
    int st;
    if (!L || !cu || !ids || !u || !keep || !out || !count) return fail(W4A8_ERR_NULL, "draft_verify: NULL pointer");
    if (!is_type(l_type) || (Q && !is_type(q_type))) return fail(W4A8_ERR_SHAPE, "draft_verify: unknown type");
    if ((st = check_vocab("draft_verify", tokens, vocab)) != W4A8_OK) return st;
    if (seqs < 1 || seqs > 65536) return fail(W4A8_ERR_SHAPE, "draft_verify: seqs=%lld outside [1, 65536]", (long long)seqs);
    if (ld_l < vocab || (Q && ld_q < vocab)) return fail(W4A8_ERR_SHAPE, "draft_verify: rows are less than vocab apart");
    if (!aligned(L, size_of(l_type)) || (Q && !aligned(Q, size_of(q_type))) || !aligned(cu, 4) || !aligned(ids, 4) ||
        !aligned(mask, 8) || !aligned(temp, 4) || !aligned(u, 4) || !aligned(keep, 4) || !aligned(out, 4) ||
        !aligned(count, 4))
        return fail(W4A8_ERR_ALIGN, "draft_verify: an array is not aligned to its element");
    if ((st = check_flags("draft_verify", flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    if ((st = check_workspace("draft_verify", ws, ws_bytes, w4a8::draft_verify_workspace(tokens, vocab, sms))) != W4A8_OK)
        return st;
    return w4a8::status_done(
        w4a8::launch_draft_verify(L, l_type, ld_l, vocab, cu, seqs, tokens, ids, mask, Q, q_type, ld_q, temp, u, keep, out,
                                  count, ws, sms, flags, st_of(stream)),
        "draft_verify launch");
}

int f8_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* Wf, float* sw, void* stream) {
    if (!W || !Wf || !sw) return fail(W4A8_ERR_NULL, "f8_quantize_weights: NULL pointer");
    int st;
    if ((st = check_linear("f8_quantize_weights", 1, K, N)) != W4A8_OK) return st;
    if (blocks(N) * blocks(K) > kIntMax) return fail(W4A8_ERR_SHAPE, "f8_quantize_weights: more than 2^31-1 blocks");
    if (!aligned(W, 16) || !aligned(Wf, 16) || !aligned(sw, 4))
        return fail(W4A8_ERR_ALIGN, "f8_quantize_weights: W and Wf need 16-byte, sw 4-byte alignment");
    return w4a8::status_done(w4a8::launch_f8_quantize_weights(W, N, K, Wf, sw, st_of(stream)), "f8_quantize_weights launch");
}

int f8_quantize_rows(const void* X, int x_type, int64_t M, int64_t K, uint8_t* Xf, float* sa, unsigned flags,
                     void* stream) {
    if (!X || !Xf || !sa) return fail(W4A8_ERR_NULL, "f8_quantize_rows: NULL pointer");
    if (!is_type(x_type)) return fail(W4A8_ERR_SHAPE, "f8_quantize_rows: unknown type");
    int st;
    if ((st = check_linear("f8_quantize_rows", M, K, 1)) != W4A8_OK) return st;
    if (!aligned(X, 16) || !aligned(Xf, 16) || !aligned(sa, 4))
        return fail(W4A8_ERR_ALIGN, "f8_quantize_rows: X and Xf need 16-byte, sa 4-byte alignment");
    if ((st = check_flags("f8_quantize_rows", flags)) != W4A8_OK) return st;
    return w4a8::status_done(w4a8::launch_f8_quantize_rows(X, x_type, M, K, Xf, sa, flags, st_of(stream)),
                             "f8_quantize_rows launch");
}

int f8_gemm(const uint8_t* Xf, const float* sa, int64_t M, int64_t K, const uint8_t* Wf, const float* sw, int64_t N,
            void* Y, int y_type, unsigned flags, void* stream) {
    if (!Xf || !sa || !Wf || !sw || !Y) return fail(W4A8_ERR_NULL, "f8_gemm: NULL pointer");
    if (!is_type(y_type)) return fail(W4A8_ERR_SHAPE, "f8_gemm: unknown type");
    int st;
    if ((st = check_linear("f8_gemm", M, K, N)) != W4A8_OK) return st;
    if (!aligned(Xf, 16) || !aligned(Wf, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(Y, size_of(y_type)))
        return fail(W4A8_ERR_ALIGN, "f8_gemm: Xf and Wf need 16-byte, the others their element's alignment");
    if ((st = check_flags("f8_gemm", flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    return w4a8::status_done(w4a8::launch_f8_gemm(Xf, sa, M, K, Wf, sw, N, Y, y_type, sms, flags, st_of(stream)),
                             "f8_gemm launch");
}

size_t f8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    return check_linear("f8_linear", M, K, N) == W4A8_OK ? linear_bytes(M, K) : 0;
}

int f8_linear(const void* X, int x_type, int64_t M, int64_t K, const uint8_t* Wf, const float* sw, int64_t N, void* Y,
              int y_type, void* ws, size_t ws_bytes, unsigned flags, void* stream) {
    if (!X || !Wf || !sw || !Y) return fail(W4A8_ERR_NULL, "f8_linear: NULL pointer");
    if (!is_type(x_type) || !is_type(y_type)) return fail(W4A8_ERR_SHAPE, "f8_linear: unknown type");
    int st;
    if ((st = check_linear("f8_linear", M, K, N)) != W4A8_OK) return st;
    if (!aligned(X, 16) || !aligned(Wf, 16) || !aligned(sw, 4) || !aligned(Y, size_of(y_type)))
        return fail(W4A8_ERR_ALIGN, "f8_linear: X and Wf need 16-byte, the others their element's alignment");
    if ((st = check_flags("f8_linear", flags)) != W4A8_OK) return st;
    int sms = 0;
    if ((st = w4a8::status_sm_count(&sms)) != W4A8_OK) return st;
    if ((st = check_workspace("f8_linear", ws, ws_bytes, linear_bytes(M, K))) != W4A8_OK) return st;
    uint8_t* Xf = static_cast<uint8_t*>(ws);
    float* sa = reinterpret_cast<float*>(Xf + linear_scales_at(M, K));
    return w4a8::status_done(
        w4a8::launch_f8_linear(X, x_type, M, K, Wf, sw, N, Y, y_type, Xf, sa, sms, flags, st_of(stream)), "f8_linear launch");
}

}  // extern "C"
