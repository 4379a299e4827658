// Attention with grouped heads over the paged cache: which of its two kernels a call takes.
#include "heads.cuh"

namespace mtpspec {
namespace {

// How a call goes.  heads_chunk.cu takes any: its units of 128 rows keep up with the cache's bytes
// even where a row of the batch has a token and a key head eight queries.  Where heads have at most 64
// elements, a tile of keys is 32 KB, and the smaller units of heads_few.cu, two CTAs an SM, get from tile
// to tile faster: up to 32 rows of work a row of the batch and key head (64 rows, a window of 1024,
// pages of 16: 43 us, not 49; 2000-4000 keys 102, not 107; from two units a row on its bytes double).
// Heads of 128 elements take the same time in both (256 rows x 4 tokens 378 and 378 us; 256 rows of
// 50-1000 keys in pages of 16 106 here, 143 there), heads of 256 133 here and 202 there.
bool few(int64_t B, int64_t Tq, int32_t Hq, int32_t Hkv, int32_t D) {
    return D <= 64 && Tq * (Hq / Hkv) <= 32 * B;
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

// What either kernel needs, so that a workspace for a batch is one for any smaller batch too, whichever
// kernel that takes.
size_t heads_attn_workspace_bytes(int32_t D) {
    const size_t chunk = heads_chunk_workspace_bytes(D), few = heads_few_workspace_bytes();
    return D <= 64 && few > chunk ? few : chunk;
}

cudaError_t run_heads_attn(const HeadsAttnArgs &a, int dtype, cudaStream_t stream) {
    return few(a.B, a.Tq, a.Hq, a.Hkv, a.D) ? run_heads_few(a, dtype, stream) : run_heads_chunk(a, dtype, stream);
}

}  // namespace mtpspec
