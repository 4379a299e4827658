// The C ABI of libmtpspec: argument validation and launches on the caller's stream.
// Declarations, argument meanings and sources are in include/libmtpspec.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "../../include/libmtpspec.h"
#include "kernels.h"

#define MTPSPEC_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kMaxV = 2147483647;  // ids are int32
constexpr int32_t kMaxD = 64;
constexpr int64_t kMaxRows = 2147483647 / (65 * 16);  // units x cluster CTAs fit a grid
constexpr int64_t kMaxH = 65536;
constexpr int64_t kMaxTokens = 1 << 20;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem_size(int dtype) { return dtype == MTPSPEC_F32 ? 4 : 2; }

// Make the stream's device current for this library's runtime and check that it is an
// sm_103 part.  Called only after every host-side check has passed.  A stream that is
// being captured into a graph must not be asked for its device (the query invalidates
// the capture); the capturing thread's current device is used then.
int prepare_device(cudaStream_t stream) {
    int dev = -1;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (stream != nullptr && cudaStreamIsCapturing(stream, &cs) != cudaSuccess) return MTPSPEC_ERR_CUDA;
    if (stream != nullptr && cs == cudaStreamCaptureStatusNone) {
        if (cudaStreamGetDevice(stream, &dev) != cudaSuccess) return MTPSPEC_ERR_CUDA;
        int cur = -1;
        if (cudaGetDevice(&cur) != cudaSuccess) return MTPSPEC_ERR_CUDA;
        if (cur != dev && cudaSetDevice(dev) != cudaSuccess) return MTPSPEC_ERR_CUDA;
    } else if (cudaGetDevice(&dev) != cudaSuccess) {
        return MTPSPEC_ERR_CUDA;
    }
    static std::mutex mu;
    static int checked[64] = {0};  // 0 unknown, 1 ok, -1 unsupported
    if (dev < 0 || dev >= 64) return MTPSPEC_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (checked[dev] == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return MTPSPEC_ERR_CUDA;
        checked[dev] = (major == 10 && minor == 3) ? 1 : -1;
    }
    return checked[dev] == 1 ? MTPSPEC_OK : MTPSPEC_ERR_UNSUPPORTED;
}

int launched(cudaError_t e) { return e == cudaSuccess ? MTPSPEC_OK : MTPSPEC_ERR_CUDA; }

}  // namespace

namespace mtpspec {
std::atomic<unsigned long long> g_launches{0};
void count_launches(int n) { g_launches.fetch_add(static_cast<unsigned long long>(n)); }
}  // namespace mtpspec

MTPSPEC_API int mtpspec_selftest_wait_timeout(int which, uint32_t limit, int32_t *status,
                                              void *stream) {
    if (which < 0 || which > 2) return MTPSPEC_ERR_ARG;
    if (limit < 1 || limit > (1u << 20)) return MTPSPEC_ERR_ARG;
    if (!status || !aligned(status, 4)) return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    cudaError_t e = which == 0 ? mtpspec::run_wait_selftest_clusters(limit, status, s)
                    : which == 1 ? mtpspec::run_wait_selftest_chunks(limit, status, s)
                                 : mtpspec::run_wait_selftest_gemm(limit, status, s);
    if (which == 2 && e == cudaSuccess) e = mtpspec::run_wait_selftest_latent_attn(limit, status, s);
    if (which == 2 && e == cudaSuccess) e = mtpspec::run_wait_selftest_latent_prefill(limit, status, s);
    return launched(e);
}

MTPSPEC_API uint64_t mtpspec_launch_count(void) {
    return static_cast<uint64_t>(mtpspec::g_launches.load());
}

MTPSPEC_API const char *mtpspec_status_string(int code) {
    switch (code) {
    case MTPSPEC_OK: return "MTPSPEC_OK";
    case MTPSPEC_ERR_ARG: return "MTPSPEC_ERR_ARG: invalid argument";
    case MTPSPEC_ERR_DTYPE: return "MTPSPEC_ERR_DTYPE: unsupported dtype";
    case MTPSPEC_ERR_SHAPE: return "MTPSPEC_ERR_SHAPE: size out of the supported range";
    case MTPSPEC_ERR_WORKSPACE: return "MTPSPEC_ERR_WORKSPACE: workspace missing or too small";
    case MTPSPEC_ERR_CUDA: return "MTPSPEC_ERR_CUDA: CUDA runtime or launch failure";
    case MTPSPEC_ERR_UNSUPPORTED: return "MTPSPEC_ERR_UNSUPPORTED: device is not sm_103";
    default: return "MTPSPEC: unknown status";
    }
}

MTPSPEC_API int mtp_greedy_draft(const void *logits, int dtype, int64_t M, int64_t V,
                                 int32_t *out_ids, void *stream) {
    if (dtype != MTPSPEC_F32 && dtype != MTPSPEC_BF16) return MTPSPEC_ERR_DTYPE;
    if (M < 0 || V < 1 || V > kMaxV || M > 2147483647 / 16) return MTPSPEC_ERR_SHAPE;
    if (M == 0) return MTPSPEC_OK;
    if (!logits || !out_ids) return MTPSPEC_ERR_ARG;
    if (!aligned(logits, elem_size(dtype)) || !aligned(out_ids, 4)) return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    return launched(mtpspec::run_greedy_draft(logits, dtype, M, V, out_ids, s));
}

MTPSPEC_API int spec_verify_greedy(const void *target_logits, int dtype, const int32_t *draft_ids,
                                   int64_t B, int32_t D, int64_t V, int32_t *out_tokens,
                                   int32_t *num_accepted, int32_t *status, void *stream) {
    if (dtype != MTPSPEC_F32 && dtype != MTPSPEC_BF16) return MTPSPEC_ERR_DTYPE;
    if (B < 0 || D < 1 || D > kMaxD || V < 1 || V > kMaxV || B > 2147483647 / 16)
        return MTPSPEC_ERR_SHAPE;
    if (B == 0) return MTPSPEC_OK;
    if (!target_logits || !draft_ids || !out_tokens || !num_accepted) return MTPSPEC_ERR_ARG;
    if (!aligned(target_logits, elem_size(dtype)) || !aligned(draft_ids, 4) ||
        !aligned(out_tokens, 4) || !aligned(num_accepted, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    return launched(mtpspec::run_verify_greedy(target_logits, dtype, draft_ids, B, D, V, out_tokens,
                                               num_accepted, status, s));
}

MTPSPEC_API size_t spec_verify_workspace_bytes(int64_t B, int32_t D, int64_t V) {
    if (B <= 0 || D < 1 || D > kMaxD || V < 1 || V > kMaxV || B > kMaxRows) return 0;
    if (!mtpspec::verify_sample_fits(V, 2, true)) return 0;  // too large for any type and mode
    return mtpspec::verify_workspace_bytes(B, D, V);
}

MTPSPEC_API int spec_verify_sample(const void *target_logits, const void *draft_logits, int dtype,
                                   const int32_t *draft_ids, const float *temperature,
                                   const int32_t *top_k, const float *top_p, uint64_t seed,
                                   int64_t B, int32_t D, int64_t V, int32_t *out_tokens,
                                   int32_t *num_accepted, float *p_target, float *p_draft,
                                   void *workspace, size_t workspace_bytes, int32_t *status,
                                   void *stream) {
    if (dtype != MTPSPEC_F32 && dtype != MTPSPEC_BF16) return MTPSPEC_ERR_DTYPE;
    if (B < 0 || D < 1 || D > kMaxD || V < 1 || V > kMaxV || B > kMaxRows) return MTPSPEC_ERR_SHAPE;
    if (!mtpspec::verify_sample_fits(V, elem_size(dtype), draft_logits == nullptr))
        return MTPSPEC_ERR_SHAPE;
    if (B == 0) return MTPSPEC_OK;
    if (!target_logits || !draft_ids || !temperature || !out_tokens || !num_accepted)
        return MTPSPEC_ERR_ARG;
    const size_t es = elem_size(dtype);
    if (!aligned(target_logits, es) || !aligned(draft_logits, es) || !aligned(draft_ids, 4) ||
        !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(out_tokens, 4) || !aligned(num_accepted, 4) || !aligned(p_target, 4) ||
        !aligned(p_draft, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < mtpspec::verify_workspace_bytes(B, D, V))
        return MTPSPEC_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::VerifySampleArgs a;
    a.target = target_logits;
    a.draft = draft_logits;
    a.dtype = dtype;
    a.draft_ids = draft_ids;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.seed = seed;
    a.B = B;
    a.D = D;
    a.V = V;
    a.out_tokens = out_tokens;
    a.num_accepted = num_accepted;
    a.p_target = p_target;
    a.p_draft = p_draft;
    a.workspace = workspace;
    a.status = status;
    return launched(mtpspec::run_verify_sample(a, s));
}

MTPSPEC_API size_t mtp_draft_input_workspace_bytes(int64_t M, int64_t H) {
    if (M <= 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens) return 0;
    return mtpspec::draft_input_workspace_bytes(M, H);
}

MTPSPEC_API int mtp_draft_input(const void *emb_next, const void *hidden, const void *enorm_w,
                                const void *hnorm_w, const void *eh_proj_w, void *out, int64_t M,
                                int64_t H, float eps, void *workspace, size_t workspace_bytes,
                                void *stream) {
    if (M < 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens) return MTPSPEC_ERR_SHAPE;
    if (!(eps >= 0.0f)) return MTPSPEC_ERR_ARG;
    if (M == 0) return MTPSPEC_OK;
    if (!emb_next || !hidden || !enorm_w || !hnorm_w || !eh_proj_w || !out) return MTPSPEC_ERR_ARG;
    if (!aligned(emb_next, 16) || !aligned(hidden, 16) || !aligned(enorm_w, 16) ||
        !aligned(hnorm_w, 16) || !aligned(eh_proj_w, 16) || !aligned(out, 16))
        return MTPSPEC_ERR_ARG;
    const size_t need = mtpspec::draft_input_workspace_bytes(M, H);
    if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
        return MTPSPEC_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::DraftInputArgs a;
    a.e = emb_next;
    a.h = hidden;
    a.we = enorm_w;
    a.wh = hnorm_w;
    a.W = eh_proj_w;
    a.y = out;
    a.M = M;
    a.H = H;
    a.eps = eps;
    a.workspace = workspace;
    return launched(mtpspec::run_draft_input(a, s));
}

constexpr int64_t kMaxLmHeadV = 65535LL * 128;  // ids stay well inside int32 tile arithmetic

MTPSPEC_API size_t mtp_lm_head_greedy_workspace_bytes(int64_t M, int64_t H, int64_t V) {
    if (M <= 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens || V < 1 || V > kMaxLmHeadV)
        return 0;
    return mtpspec::lm_head_workspace_bytes(M, H, V);
}

MTPSPEC_API int mtp_lm_head_greedy(const void *hidden, const void *norm_w, float eps,
                                   const void *lm_head_w, int64_t M, int64_t H, int64_t V,
                                   int32_t *out_ids, float *out_logit, void *workspace,
                                   size_t workspace_bytes, int32_t *status, void *stream) {
    if (M < 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens || V < 1 || V > kMaxLmHeadV)
        return MTPSPEC_ERR_SHAPE;
    if (!(eps >= 0.0f)) return MTPSPEC_ERR_ARG;
    if (M == 0) return MTPSPEC_OK;
    if (!hidden || !lm_head_w || !out_ids) return MTPSPEC_ERR_ARG;
    if (!aligned(hidden, 16) || !aligned(norm_w, 16) || !aligned(lm_head_w, 16) ||
        !aligned(out_ids, 4) || !aligned(out_logit, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < mtpspec::lm_head_workspace_bytes(M, H, V))
        return MTPSPEC_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::LmHeadArgs a;
    a.hidden = hidden;
    a.norm_w = norm_w;
    a.eps = eps;
    a.W = lm_head_w;
    a.M = M;
    a.H = H;
    a.V = V;
    a.ids = out_ids;
    a.ids_stride = 1;
    a.logit = out_logit;
    a.k = 1;
    a.workspace = workspace;
    a.status = status;
    return launched(mtpspec::run_lm_head_greedy(a, s));
}

MTPSPEC_API size_t mtp_draft_steps_workspace_bytes(int64_t M, int64_t H, int64_t V) {
    if (M <= 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens || V < 1 || V > kMaxLmHeadV)
        return 0;
    return mtpspec::draft_steps_workspace_bytes(M, H, V);
}

MTPSPEC_API int mtp_draft_steps(const void *embed_w, const int32_t *next_ids, const int32_t *positions,
                                const void *hidden, const void *enorm_w, const void *hnorm_w,
                                const void *eh_proj_w, const void *norm_w, const void *lm_head_w,
                                float eps, int64_t M, int64_t H, int64_t V, int32_t D,
                                int32_t *draft_ids, void *hidden_out, void *workspace,
                                size_t workspace_bytes, int32_t *status, void *stream) {
    if (M < 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens || V < 1 || V > kMaxLmHeadV ||
        D < 1 || D > kMaxD)
        return MTPSPEC_ERR_SHAPE;
    if (!(eps >= 0.0f)) return MTPSPEC_ERR_ARG;
    if (M == 0) return MTPSPEC_OK;
    if (!embed_w || !next_ids || !hidden || !enorm_w || !hnorm_w || !eh_proj_w || !lm_head_w ||
        !draft_ids)
        return MTPSPEC_ERR_ARG;
    if (!aligned(embed_w, 16) || !aligned(hidden, 16) || !aligned(enorm_w, 16) ||
        !aligned(hnorm_w, 16) || !aligned(eh_proj_w, 16) || !aligned(norm_w, 16) ||
        !aligned(lm_head_w, 16) || !aligned(hidden_out, 16) || !aligned(next_ids, 4) ||
        !aligned(positions, 4) || !aligned(draft_ids, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < mtpspec::draft_steps_workspace_bytes(M, H, V))
        return MTPSPEC_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::DraftStepsArgs a;
    a.embed = embed_w;
    a.next_ids = next_ids;
    a.positions = positions;
    a.hidden = hidden;
    a.enorm_w = enorm_w;
    a.hnorm_w = hnorm_w;
    a.eh_proj_w = eh_proj_w;
    a.norm_w = norm_w;
    a.lm_head_w = lm_head_w;
    a.eps = eps;
    a.M = M;
    a.H = H;
    a.V = V;
    a.D = D;
    a.draft_ids = draft_ids;
    a.hidden_out = hidden_out;
    a.workspace = workspace;
    a.status = status;
    return launched(mtpspec::run_draft_steps(a, s));
}

MTPSPEC_API size_t mtp_lm_head_topk_workspace_bytes(int64_t M, int64_t H, int64_t V) {
    if (M <= 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens || V < 1 || V > kMaxLmHeadV)
        return 0;
    return mtpspec::lm_head_workspace_bytes(M, H, V, mtpspec::kLmHeadTopK);
}

MTPSPEC_API int mtp_lm_head_topk(const void *hidden, const void *norm_w, float eps,
                                 const void *lm_head_w, int64_t M, int64_t H, int64_t V, int32_t k,
                                 int32_t *out_ids, float *out_logits, void *workspace,
                                 size_t workspace_bytes, int32_t *status, void *stream) {
    if (M < 0 || H < 8 || H > kMaxH || (H % 8) != 0 || M > kMaxTokens || V < 1 || V > kMaxLmHeadV)
        return MTPSPEC_ERR_SHAPE;
    if (k < 1 || k > mtpspec::kLmHeadTopK || k > V) return MTPSPEC_ERR_SHAPE;
    if (!(eps >= 0.0f)) return MTPSPEC_ERR_ARG;
    if (M == 0) return MTPSPEC_OK;
    if (!hidden || !lm_head_w || !out_ids) return MTPSPEC_ERR_ARG;
    if (!aligned(hidden, 16) || !aligned(norm_w, 16) || !aligned(lm_head_w, 16) ||
        !aligned(out_ids, 4) || !aligned(out_logits, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < mtpspec::lm_head_workspace_bytes(M, H, V, mtpspec::kLmHeadTopK))
        return MTPSPEC_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::LmHeadArgs a;
    a.hidden = hidden;
    a.norm_w = norm_w;
    a.eps = eps;
    a.W = lm_head_w;
    a.M = M;
    a.H = H;
    a.V = V;
    a.ids = out_ids;
    a.ids_stride = k;
    a.logit = out_logits;
    a.k = k;  // k = 1 is the greedy pick, with the same layout of ids and logits
    a.workspace = workspace;
    a.status = status;
    return launched(mtpspec::run_lm_head_greedy(a, s));
}

constexpr int64_t kMaxStateRows = 1LL << 24;

MTPSPEC_API int mtp_state_snapshot(const void *state, void *backup, int64_t B, int64_t row_bytes,
                                   void *stream) {
    if (B < 0 || B > kMaxStateRows || row_bytes < 0 || (row_bytes % 16) != 0) return MTPSPEC_ERR_SHAPE;
    if (B == 0 || row_bytes == 0) return MTPSPEC_OK;
    if (!state || !backup || !aligned(state, 16) || !aligned(backup, 16)) return MTPSPEC_ERR_ARG;
    const char *s0 = static_cast<const char *>(state), *b0 = static_cast<const char *>(backup);
    const int64_t n = B * row_bytes;
    if (s0 < b0 + n && b0 < s0 + n) return MTPSPEC_ERR_ARG;  // overlapping
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    return launched(mtpspec::run_state_snapshot(state, backup, B, row_bytes, s));
}

MTPSPEC_API int mtp_state_fixup(const int32_t *num_accepted, int32_t D, const int32_t *kv_len_before,
                                int32_t *kv_len, void *state, const void *backup, int64_t B,
                                int64_t row_bytes, int32_t *draft_kv_len, int32_t *recompute,
                                int32_t *status, void *stream) {
    if (B < 0 || B > kMaxStateRows || D < 1 || D > kMaxD || row_bytes < 0 || (row_bytes % 16) != 0)
        return MTPSPEC_ERR_SHAPE;
    if (B == 0) return MTPSPEC_OK;
    if (!num_accepted || !kv_len_before || !kv_len) return MTPSPEC_ERR_ARG;
    if (!aligned(num_accepted, 4) || !aligned(kv_len_before, 4) || !aligned(kv_len, 4) ||
        !aligned(draft_kv_len, 4) || !aligned(recompute, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    if (row_bytes > 0) {
        if (!state || !backup || !aligned(state, 16) || !aligned(backup, 16)) return MTPSPEC_ERR_ARG;
        const char *s0 = static_cast<const char *>(state), *b0 = static_cast<const char *>(backup);
        const int64_t n = B * row_bytes;
        if (s0 < b0 + n && b0 < s0 + n) return MTPSPEC_ERR_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    return launched(mtpspec::run_state_fixup(num_accepted, D, kv_len_before, kv_len, state, backup,
                                             B, row_bytes, draft_kv_len, recompute, status, s));
}

MTPSPEC_API int spec_verify_sample_static(const void *target_logits, const void *draft_logits,
                                          int dtype, const int32_t *draft_ids,
                                          const float *temperature, const int32_t *top_k,
                                          const float *top_p, uint64_t seed, int64_t B, int32_t D,
                                          int64_t V, int32_t *out_tokens, int32_t *num_accepted,
                                          float *p_target, float *p_draft, int32_t *status,
                                          void *stream) {
    if (dtype != MTPSPEC_F32 && dtype != MTPSPEC_BF16) return MTPSPEC_ERR_DTYPE;
    if (B < 0 || D < 1 || D > kMaxD || V < 1 || V > kMaxV || B > kMaxRows) return MTPSPEC_ERR_SHAPE;
    if (B * (D + 1) > mtpspec::kStaticVerifyUnits) return MTPSPEC_ERR_SHAPE;
    if (!mtpspec::verify_fits(V, elem_size(dtype), draft_logits == nullptr)) return MTPSPEC_ERR_SHAPE;
    if (B == 0) return MTPSPEC_OK;
    if (!target_logits || !draft_ids || !temperature || !out_tokens || !num_accepted)
        return MTPSPEC_ERR_ARG;
    const size_t es = elem_size(dtype);
    if (!aligned(target_logits, es) || !aligned(draft_logits, es) || !aligned(draft_ids, 4) ||
        !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(out_tokens, 4) || !aligned(num_accepted, 4) || !aligned(p_target, 4) ||
        !aligned(p_draft, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::VerifySampleArgs a;
    a.target = target_logits;
    a.draft = draft_logits;
    a.dtype = dtype;
    a.draft_ids = draft_ids;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.seed = seed;
    a.B = B;
    a.D = D;
    a.V = V;
    a.out_tokens = out_tokens;
    a.num_accepted = num_accepted;
    a.p_target = p_target;
    a.p_draft = p_draft;
    a.workspace = nullptr;
    a.status = status;
    return launched(mtpspec::run_verify_sample_static(a, s));
}

// ---------------------------------------------------------------- latent attention

namespace {

constexpr int64_t kMaxLatentRows = 1 << 20;
constexpr int32_t kMaxHeads = 1024;
constexpr int64_t kMaxPromptTokens = 1 << 24;
constexpr int64_t kMaxStride = (int64_t{1} << 39) - 8;  // elements: a tensor map strides below 2^40 bytes

bool is_half(int dtype) { return dtype == MTPSPEC_BF16 || dtype == MTPSPEC_F16; }
bool latent_sizes(int32_t L, int32_t R) {
    return L >= 64 && L <= 512 && L % 64 == 0 && R >= 16 && R <= 64 && R % 16 == 0;
}
bool cache_sizes(int64_t num_pages, int32_t page_size, int64_t page_stride, int64_t max_pages,
                 int32_t row) {
    return num_pages >= 1 && num_pages <= kMaxV && max_pages >= 1 && max_pages <= kMaxV &&
           page_size >= 8 && page_size <= (1 << 24) && page_size % 8 == 0 &&
           page_stride >= static_cast<int64_t>(page_size) * row && page_stride <= kMaxStride &&
           page_stride % 8 == 0;
}
// A stride over `n` items of `item` elements each: 16-byte steps, and no overlap along this axis.
bool stride_ok(int64_t stride, int64_t n, int64_t item) {
    return stride % 8 == 0 && stride <= kMaxStride && (n <= 1 ? stride >= 0 : stride >= item);
}
// An output whose items of `item` elements lie along three axes: no item overlaps another, since
// every axis steps over all that the axes of smaller strides span.  (Two writers of one element
// would leave either's value.)
bool apart(int64_t item, int64_t s0, int64_t n0, int64_t s1, int64_t n1, int64_t s2 = 0, int64_t n2 = 1) {
    int64_t s[3] = {s0, s1, s2}, n[3] = {n0, n1, n2}, span = item;
    for (int done = 0; done < 3; ++done) {
        int k = -1;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && (k < 0 || s[i] < s[k])) k = i;
        if (k < 0) break;
        if (s[k] < span) return false;
        span += s[k] * (n[k] - 1);
        n[k] = 1;
    }
    return true;
}

}  // namespace

MTPSPEC_API int mtp_latent_append(
    const void *latent, int64_t latent_stride, const void *rot, int64_t rot_stride,
    const void *norm_w, float eps, const float *cos_sin, int64_t max_pos, int32_t interleaved,
    const int32_t *tok_row, const int32_t *positions, int64_t T, int32_t L, int32_t R,
    const int32_t *block_table, int64_t B, int64_t max_pages, void *cache, int64_t num_pages,
    int32_t page_size, int64_t page_stride, const void *q_rot, int64_t q_rot_tok_stride,
    int64_t q_rot_head_stride, void *q_out, int64_t q_out_tok_stride, int64_t q_out_head_stride,
    int32_t Hq, int dtype, int32_t *status, void *stream) {
    if (!is_half(dtype)) return MTPSPEC_ERR_DTYPE;
    if (T < 0 || T > kMaxTokens || B < 1 || B > kMaxLatentRows || max_pos < 1 || max_pos > kMaxV ||
        !latent_sizes(L, R) || !cache_sizes(num_pages, page_size, page_stride, max_pages, L + R))
        return MTPSPEC_ERR_SHAPE;
    if (!stride_ok(latent_stride, T, L) || !stride_ok(rot_stride, T, R)) return MTPSPEC_ERR_SHAPE;
    const bool queries = q_rot != nullptr || q_out != nullptr;
    if (queries) {
        if (!q_rot || !q_out) return MTPSPEC_ERR_ARG;
        if (Hq < 1 || Hq > kMaxHeads || !stride_ok(q_rot_head_stride, Hq, R) ||
            !stride_ok(q_out_head_stride, Hq, R) || !stride_ok(q_rot_tok_stride, T, R) ||
            !stride_ok(q_out_tok_stride, T, R) ||
            !apart(R, q_out_tok_stride, T, q_out_head_stride, Hq))
            return MTPSPEC_ERR_SHAPE;
    }
    if (!(eps >= 0.0f)) return MTPSPEC_ERR_ARG;
    if (T == 0) return MTPSPEC_OK;
    if (!latent || !rot || !cos_sin || !tok_row || !positions || !block_table || !cache)
        return MTPSPEC_ERR_ARG;
    if (!aligned(latent, 16) || !aligned(rot, 16) || !aligned(norm_w, 16) || !aligned(cos_sin, 16) ||
        !aligned(tok_row, 4) || !aligned(positions, 4) || !aligned(block_table, 4) ||
        !aligned(cache, 16) || !aligned(q_rot, 16) || !aligned(q_out, 16) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::LatentAppendArgs a = {};
    a.latent = static_cast<const uint16_t *>(latent);
    a.rot = static_cast<const uint16_t *>(rot);
    a.norm_w = static_cast<const uint16_t *>(norm_w);
    a.latent_stride = latent_stride;
    a.rot_stride = rot_stride;
    a.eps = eps;
    a.cos_sin = cos_sin;
    a.interleaved = interleaved;
    a.tok_row = tok_row;
    a.positions = positions;
    a.T = T;
    a.L = L;
    a.R = R;
    a.block_table = block_table;
    a.B = B;
    a.max_pages = max_pages;
    const int64_t slots = max_pages * page_size;
    a.pos_end = max_pos < slots ? max_pos : slots;
    a.cache = static_cast<uint16_t *>(cache);
    a.num_pages = num_pages;
    a.page_stride = page_stride;
    a.page_size = page_size;
    a.q_rot = static_cast<const uint16_t *>(q_rot);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.q_rot_tok = q_rot_tok_stride;
    a.q_rot_head = q_rot_head_stride;
    a.q_out_tok = q_out_tok_stride;
    a.q_out_head = q_out_head_stride;
    a.Hq = Hq;
    a.status = status;
    return launched(mtpspec::run_latent_append(a, dtype, s));
}

namespace {

bool attn_sizes(int64_t B, int32_t T, int32_t Hq, int32_t L, int32_t R) {
    return B >= 0 && B <= kMaxLatentRows && T >= 1 && T <= 256 && Hq >= 1 && Hq <= kMaxHeads &&
           static_cast<int64_t>(T) * Hq <= 65536 && B * T * Hq <= kMaxV && latent_sizes(L, R);
}
bool good_scale(float s) { return s > 0.0f && s - s == 0.0f; }

}  // namespace

MTPSPEC_API size_t mtp_latent_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t L,
                                                   int32_t R) {
    if (!attn_sizes(B, T, Hq, L, R) || B == 0) return 0;
    return mtpspec::latent_attn_workspace_bytes(B, T, Hq, L);
}

MTPSPEC_API int mtp_latent_attn(const void *q, int64_t q_row_stride, int64_t q_tok_stride,
                                int64_t q_head_stride, const void *cache, int64_t num_pages,
                                int32_t page_size, int64_t page_stride, const int32_t *block_table,
                                int64_t max_pages, const int32_t *kv_len, int64_t B, int32_t T,
                                int32_t Hq, int32_t L, int32_t R, float scale, void *out,
                                int64_t out_row_stride, int64_t out_tok_stride,
                                int64_t out_head_stride, float *lse, int dtype, void *workspace,
                                size_t workspace_bytes, int32_t *status, void *stream) {
    if (!is_half(dtype)) return MTPSPEC_ERR_DTYPE;
    if (!attn_sizes(B, T, Hq, L, R) ||
        !cache_sizes(num_pages, page_size, page_stride, max_pages, L + R))
        return MTPSPEC_ERR_SHAPE;
    if (!stride_ok(q_row_stride, B, L + R) || !stride_ok(q_tok_stride, T, L + R) ||
        !stride_ok(q_head_stride, Hq, L + R) || !stride_ok(out_row_stride, B, L) ||
        !stride_ok(out_tok_stride, T, L) || !stride_ok(out_head_stride, Hq, L) ||
        !apart(L, out_row_stride, B, out_tok_stride, T, out_head_stride, Hq))
        return MTPSPEC_ERR_SHAPE;
    if (!good_scale(scale)) return MTPSPEC_ERR_ARG;
    if (B == 0) return MTPSPEC_OK;
    if (!q || !cache || !block_table || !kv_len || !out) return MTPSPEC_ERR_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(block_table, 4) || !aligned(kv_len, 4) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    if (!workspace || workspace_bytes < mtpspec::latent_attn_workspace_bytes(B, T, Hq, L))
        return MTPSPEC_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::LatentAttnArgs a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.q_row = q_row_stride;
    a.q_tok = q_tok_stride;
    a.q_head = q_head_stride;
    a.cache = static_cast<const uint16_t *>(cache);
    a.num_pages = num_pages;
    a.page_stride = page_stride;
    a.page_size = page_size;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.kv_len = kv_len;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.L = L;
    a.R = R;
    a.scale = scale;
    a.out = static_cast<uint16_t *>(out);
    a.out_row = out_row_stride;
    a.out_tok = out_tok_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.workspace = workspace;
    a.status = status;
    return launched(mtpspec::run_latent_attn(a, dtype, s));
}

MTPSPEC_API int mtp_latent_prefill(const void *q, int64_t q_tok_stride, int64_t q_head_stride,
                                   const void *kv, int64_t kv_tok_stride, int64_t kv_head_stride,
                                   const void *rot, int64_t rot_stride, const int32_t *cu_q,
                                   const int32_t *cu_k, int64_t B, int64_t Tq, int64_t Tk,
                                   int32_t Hq, int32_t N, int32_t R, int32_t V, float scale,
                                   void *out, int64_t out_tok_stride, int64_t out_head_stride,
                                   float *lse, int dtype, int32_t *status, void *stream) {
    if (!is_half(dtype)) return MTPSPEC_ERR_DTYPE;
    if (B < 1 || B > 65536 || Tq < 0 || Tq > kMaxPromptTokens || Tk < 0 || Tk > kMaxPromptTokens ||
        (Tq > 0 && Tk < 1) || Hq < 1 || Hq > kMaxHeads || (N != 64 && N != 128) ||
        (V != 64 && V != 128) || R < 16 || R > 64 || R % 16 != 0)
        return MTPSPEC_ERR_SHAPE;
    if (!stride_ok(q_tok_stride, Tq, N + R) || !stride_ok(q_head_stride, Hq, N + R) ||
        !stride_ok(kv_tok_stride, Tk, N + V) || !stride_ok(kv_head_stride, Hq, N + V) ||
        !stride_ok(rot_stride, Tk, R) || !stride_ok(out_tok_stride, Tq, V) ||
        !stride_ok(out_head_stride, Hq, V) || !apart(V, out_tok_stride, Tq, out_head_stride, Hq))
        return MTPSPEC_ERR_SHAPE;
    if (!good_scale(scale)) return MTPSPEC_ERR_ARG;
    if (Tq == 0) return MTPSPEC_OK;
    if (!q || !kv || !rot || !cu_q || !cu_k || !out) return MTPSPEC_ERR_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(rot, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(status, 4))
        return MTPSPEC_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = prepare_device(s);
    if (rc != MTPSPEC_OK) return rc;
    mtpspec::LatentPrefillArgs a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.kv = static_cast<const uint16_t *>(kv);
    a.rot = static_cast<const uint16_t *>(rot);
    a.q_tok = q_tok_stride;
    a.q_head = q_head_stride;
    a.kv_tok = kv_tok_stride;
    a.kv_head = kv_head_stride;
    a.rot_stride = rot_stride;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.Hq = Hq;
    a.N = N;
    a.R = R;
    a.V = V;
    a.scale = scale;
    a.out = static_cast<uint16_t *>(out);
    a.out_tok = out_tok_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.status = status;
    return launched(mtpspec::run_latent_prefill(a, dtype, s));
}
