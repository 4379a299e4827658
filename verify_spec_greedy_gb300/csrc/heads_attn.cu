// Attention with grouped heads over the paged cache: which of its two kernels a call takes.
#include "heads.cuh"

namespace mtpspec {
namespace {

// How a call goes.  heads_chunk.cu takes any: units of 128 rows.  Where heads have at most 64 elements,
// a tile of keys is 32 KB, and the units of 32 rows of heads_few.cu, two CTAs an SM, get from tile to
// tile faster as long as a row of the batch and key head fills one or two.  In us, heads of 64, eight key
// heads, few / chunk:
//   1 token a row, a window of 1024 and 4: 4 rows 14.4 / 15.5, 16 rows 18 / 20, 64 rows 37 / 49, 256 rows
//   131 / 154; a window of 128: 64 rows 17 / 26, 256 rows 40 / 75; 256 rows over 50-100 keys 32 / 47, over
//   500-1000 90 / 104, over 2000-4000 371 / 366; 4 tokens a row over 2000-4000 377 / 370
// (Such units for heads of 128: 4 tokens a row 378 / 378, 256 rows over 50-1000 keys 143 / 106; of 256: 202 /
// 133.)
//
// The host knows how many tokens a row has on average only.  A batch of drafts or verifications has the
// same number in every row, so its tokens are a multiple of the rows; in one that mixes prompts with
// drafts, or with rows of no tokens, each of the prompt's units of 32 rows reads all its keys:
//   a prompt of 64 / 256 / 700 / 4000 tokens in a table of 1024 rows of none: 13 / 25 / 66 / 662, in
//   heads_chunk.cu 11 / 15 / 29 / 233; of 700 beside 255 drafts over 1000 keys 167 / 140
//   256 rows of 1-4 tokens over 100-200 keys: 47 / 69, over 500-1000 91 / 105
// So other batches are taken up to the tokens that 256 such rows have, 640 and two deviations.
bool few(int64_t B, int64_t Tq, int32_t Hq, int32_t Hkv, int32_t D) {
    return D <= 64 && Tq * (Hq / Hkv) <= 32 * B && (Tq <= 680 || Tq % B == 0);
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
