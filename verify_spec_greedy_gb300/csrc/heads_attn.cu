// Attention with grouped heads over the paged cache: which of its two kernels a call takes.
#include "heads.cuh"

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

// Diagnostic of the bounded waits, as the other kernels': on a barrier of two arrivals that got one,
// both forms must give up after `limit` polls and raise the abort flag; if not, the timeout is taken
// out of the status word.
namespace heads {
struct WaitShared {
    uint64_t never;
    volatile int abort;
};
__global__ void k_wait_selftest(uint32_t limit, int32_t *status) {
    __shared__ WaitShared sh;
    if (threadIdx.x != 0) return;
    mbar_init(&sh.never, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_arrive(&sh.never);
    bool ok = true;
    for (int form = 0; form < 2; ++form) {
        sh.abort = 0;
        const bool got = form == 0 ? wait(sh, &sh.never, 0, limit) : wait_long(sh, &sh.never, 0, limit);
        ok &= !got && sh.abort;
    }
    if (!ok) atomicAnd(status, ~MTPSPEC_STATUS_TIMEOUT);
}
}  // namespace heads

cudaError_t run_wait_selftest_heads(uint32_t limit, int32_t *status, cudaStream_t stream) {
    heads::k_wait_selftest<<<1, 32, 0, stream>>>(limit, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

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
