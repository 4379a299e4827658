// Attention with grouped heads over the paged cache: which of its two kernels a call takes.
#include "kernels.h"

namespace mtpspec {
namespace {

// How a call goes.  A row has Tq / B tokens on average and G = Hq / Hkv rows of work a token and
// key head.  What fits 32 or 64 rows is bound by the cache's bytes, which heads_few.cu streams with
// few threads a row; more rows are bound by products, for which heads_chunk.cu has pairs of
// 128-row tiles.
enum class Form { few32, few64, chunk };
Form form_of(int64_t B, int64_t Tq, int32_t Hq, int32_t Hkv) {
    const int64_t rows = Tq * (Hq / Hkv);
    if (rows <= 32 * B) return Form::few32;
    return rows <= 64 * B ? Form::few64 : Form::chunk;
}

}  // namespace

size_t heads_attn_workspace_bytes(int64_t B, int64_t Tq, int32_t Hq, int32_t Hkv, int32_t D) {
    const Form f = form_of(B, Tq, Hq, Hkv);
    return f == Form::chunk ? heads_chunk_workspace_bytes(D) : heads_few_workspace_bytes(D, f == Form::few32);
}

cudaError_t run_heads_attn(const HeadsAttnArgs &a, int dtype, cudaStream_t stream) {
    const Form f = form_of(a.B, a.Tq, a.Hq, a.Hkv);
    return f == Form::chunk ? run_heads_chunk(a, dtype, stream)
                            : run_heads_few(a, f == Form::few32, dtype, stream);
}

}  // namespace mtpspec
