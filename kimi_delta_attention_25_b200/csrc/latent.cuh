// latent.cuh -- what the latent attention's kernels share: the problem's description, the sequences'
// offsets, and the checks of both.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// The expanded form: q [tokens, H, 128 + R] and out [tokens, H, 128] dense; k and v [keys, H, 128] with
// strides (they may be views of one up-projection), k_shared [keys, R] with a row stride, R = 64 or 0.
struct LatentArgs {
    const __nv_bfloat16 *q, *k, *v, *r;
    long long k_tok, k_head, v_tok, v_head, r_tok;   // strides in elements
    const int32_t *cu_q, *cu_k;                      // null: B sequences of T queries and Tk keys
    __nv_bfloat16 *out;
    float *lse;
    int B, T, Tk, H, N, R, causal;
    float scale;
    int32_t *status;
};

struct LatentSpan { long long q0, q1, k0, k1; };

// Sequence n's queries [q0, q1) and keys [k0, k1). False for offsets that lie outside the tensors.
__device__ __forceinline__ bool latent_span(const int32_t *cu_q, const int32_t *cu_k, int n, int T, int Tk, LatentSpan *s)
{
    if (cu_q) { s->q0 = cu_q[n]; s->q1 = cu_q[n + 1]; }
    else { s->q0 = (long long)n * T; s->q1 = s->q0 + T; }
    if (cu_k) { s->k0 = cu_k[n]; s->k1 = cu_k[n + 1]; }
    else { s->k0 = (long long)n * Tk; s->k1 = s->k0 + Tk; }
    if (cu_q && (s->q0 < 0 || s->q1 < s->q0 || s->q1 > T)) return false;
    if (cu_k && (s->k0 < 0 || s->k1 < s->k0 || s->k1 > Tk)) return false;
    return true;
}

// The sequence that holds token `tok` of offsets `cu` (or of B rows of T tokens), by bisection; -1 if none does.
__device__ __forceinline__ int latent_sequence(const int32_t *cu, int N, int T, long long tok)
{
    if (!cu) return (int)((uint32_t)tok / (uint32_t)T);       // B T tokens are below 2^31
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= tok) lo = mid; else hi = mid - 1;
    }
    return (cu[lo] <= tok && tok < cu[lo + 1]) ? lo : -1;
}

// Tile c of sequence n over offsets `cu` (rows of `tile`) has slot floor(first row / tile) + n + c: unique, and
// below total / tile + N. The inverse: the sequence and the tile's first row within it; false for a slot that no
// tile uses, and for offsets that lie outside the tensors. Called by whole warps.
__device__ __forceinline__ bool latent_slot(const int32_t *cu, const LatentArgs &a, int L, bool keys, int tile, long long slot,
                                            int *n, LatentSpan *s, long long *row)
{
    // the last sequence whose first slot is not behind `slot`: the warp's lanes ask for 32 of them at a time
    const int lane = threadIdx.x & 31;
    int lo = 0, count = a.N;
    while (count > 1) {
        const int step = (count + 31) / 32, at = lo + lane * step;
        const long long st = at < lo + count ? (cu ? (long long)cu[at] : (long long)at * L) : 0;
        const uint32_t before = __ballot_sync(0xffffffffu, at < lo + count && st / tile + at <= slot);
        const int i = before ? 31 - __clz(before) : 0;         // offsets that decrease give some sequence, checked below
        count = min(step, count - i * step);
        lo += i * step;
    }
    if (!latent_span(a.cu_q, a.cu_k, lo, a.T, a.Tk, s)) return false;
    const long long first = keys ? s->k0 : s->q0, rows = keys ? s->k1 - s->k0 : s->q1 - s->q0;
    const long long c = slot - (first / tile + lo);
    if (c < 0 || c * tile >= rows) return false;
    *n = lo;
    *row = c * tile;
    return true;
}

// The query tile (of `tile` rows) whose row of key tiles is the rank-th longest, of packed sequences, where the slots'
// order says nothing about it: with few blocks to an SM the last ones should be the shortest. Every block counts for
// itself, a time that grows with the square of the slots, so only up to kRankedSlots slots. Ranked and in slot order, 4 and
// 16 heads: 60 slots behind histories of up to 1500 keys 31 and 44 us, 109 and 115 us (9 sequences of some 300 queries
// behind histories, 16 heads: 75 and 88), prompts of up to 50 tokens 17 and 16 us, 55 and 50 us; 122 slots 63 and 69,
// 242 and 231 behind histories, 34 and 29, 111 and 97 for prompts; 375 slots 257 and 179, 999 and 658, and 167 and 73, 665 and
// 291 for prompts. All of the block's threads; `scratch` is shared memory for 2 slots + 1 integers, which the caller may use
// again when this returns (bulk copies: behind a proxy fence).
constexpr int kRankedSlots = 64;
__device__ __forceinline__ bool latent_ranked(const LatentArgs &a, int tile, int slots, int rank, int *scratch, LatentSpan *s,
                                              long long *row)
{
    int *work = scratch, *seq = scratch + slots, *found = seq + slots;
    for (int i = threadIdx.x; i < slots; i += blockDim.x) work[i] = -1;
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int n = threadIdx.x; n < a.N; n += blockDim.x) {
        LatentSpan x;
        if (!latent_span(a.cu_q, a.cu_k, n, a.T, a.Tk, &x)) continue;
        const long long Lq = x.q1 - x.q0, Lk = x.k1 - x.k0;
        for (long long c = 0; c * tile < Lq; ++c) {
            const long long i = x.q0 / tile + n + c, keys = a.causal ? min(Lk, min((c + 1) * tile, Lq) + Lk - Lq) : Lk;
            if (i < slots) { work[i] = keys > 0 ? (int)((keys + 127) / 128) : 0; seq[i] = n; }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += blockDim.x) {
        const int w = work[i];
        int r = 0;
        if (w >= 0) {
            for (int j = 0; j < slots; ++j) r += work[j] > w || (work[j] == w && j < i);
            if (r == rank) *found = i;
        }
    }
    __syncthreads();
    const int slot = *found, n = slot >= 0 ? seq[slot] : 0;
    __syncthreads();
    if (slot < 0 || !latent_span(a.cu_q, a.cu_k, n, a.T, a.Tk, s)) return false;
    *row = (slot - (s->q0 / tile + n)) * tile;
    return *row >= 0 && *row < s->q1 - s->q0;
}

// Records offsets that break the contract (cu[0] = 0, non-decreasing, cu[N] = T). One block's threads.
__device__ __forceinline__ void check_offsets(const int32_t *cu, int N, int T, int32_t *status)
{
    if (!cu) return;
    for (int n = threadIdx.x; n < N; n += blockDim.x) {
        const int a = cu[n], b = cu[n + 1];
        if ((n == 0 && a != 0) || b < a || b > T || a < 0 || (n == N - 1 && b != T)) set_status(status, KDA_ERR_INVALID_ARG);
    }
}

// Clears the status word and checks both offset arrays: the first block of a call's first kernel, all its threads.
__device__ __forceinline__ void check_call(const LatentArgs &a)
{
    if (threadIdx.x == 0) *a.status = KDA_OK;
    __syncthreads();
    check_offsets(a.cu_q, a.N, a.T, a.status);
    check_offsets(a.cu_k, a.N, a.Tk, a.status);
}

// Host checks of the expanded form's arguments, and the description they give.
kda_status_t check_latent(const void *q, const void *k, const void *v, const void *k_shared, const int32_t *cu_q,
                          const int32_t *cu_k, const void *out, const float *lse, int B, int T, int Tk, int H, int N,
                          int dk, int dv, int dr, long long k_tok, long long k_head, long long v_tok, long long v_head,
                          long long r_tok, float scale, kda_dtype_t dtype, const void *workspace, size_t workspace_bytes,
                          size_t need, LatentArgs *a);

cudaError_t launch_latent_fwd(const LatentArgs &a, cudaStream_t stream);
// A call without work: its status word, cleared or with what the offsets break.
cudaError_t launch_latent_check(const LatentArgs &a, cudaStream_t stream);

struct LatentBwdArgs {
    const __nv_bfloat16 *dout;
    __nv_bfloat16 *dq, *dk, *dv, *dr;     // dense
    float *stat;                          // [2][H][tokens]: lse in the log2 domain (+infinity for empty rows), dout . out
    float *dr_head;                       // [keys, H, R]: each head's part of the shared key's gradient
};
cudaError_t launch_latent_bwd(const LatentArgs &a, const LatentBwdArgs &b, cudaStream_t stream);

}  // namespace kda
