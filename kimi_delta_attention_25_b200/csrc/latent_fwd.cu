// latent_fwd.cu -- the expanded form of the latent attention: softmax attention whose keys are a part
// per head (128 channels, expanded from the token's latent vector) and a part that all heads share (64
// channels, or none):  s_ij = scale (q_i[:128] . k_j + q_i[128:] . r_j),  o_i = sum_j softmax_j(s_ij) v_j.
// Packed sequences with their own numbers of queries and keys; with `causal` query i of Lq sees the keys
// up to i + Lk - Lq.
#include "latent.cuh"

namespace kda {
namespace {

// One warp per (query, head): the running maximum and sum over the keys, fp32 throughout.
__global__ void __launch_bounds__(128) latent_fwd_simple(LatentArgs a)
{
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        check_offsets(a.cu_q, a.N, a.T, a.status);
        check_offsets(a.cu_k, a.N, a.Tk, a.status);
    }
    const long long tok = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = blockIdx.y, lane = threadIdx.x & 31;
    if (tok >= (long long)a.B * a.T) return;
    const int n = latent_sequence(a.cu_q, a.N, a.T, tok);
    LatentSpan s;
    if (n < 0 || !latent_span(a.cu_q, a.cu_k, n, a.T, a.Tk, &s)) return;
    const int W = kHeadDim + a.R;
    const __nv_bfloat16 *q = a.q + ((size_t)tok * a.H + h) * W;
    float qv[6] = {}, acc[4] = {};
    for (int c = 0; c < W / 32; ++c) qv[c] = to_f32(q[c * 32 + lane]);
    float m = -INFINITY, l = 0.f;
    const long long hi = a.causal ? min(s.k1 - s.k0, tok - s.q0 + (s.k1 - s.k0) - (s.q1 - s.q0) + 1) : s.k1 - s.k0;
    for (long long j = 0; j < hi; ++j) {
        const __nv_bfloat16 *k = a.k + (s.k0 + j) * a.k_tok + h * a.k_head, *v = a.v + (s.k0 + j) * a.v_tok + h * a.v_head;
        float d = 0.f;
        for (int c = 0; c < 4; ++c) d += qv[c] * to_f32(k[c * 32 + lane]);
        if (a.R) for (int c = 0; c < 2; ++c) d += qv[4 + c] * to_f32(a.r[(s.k0 + j) * a.r_tok + c * 32 + lane]);
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        d *= a.scale;
        const float m2 = fmaxf(m, d);
        if (m2 == -INFINITY) continue;
        const float f = expf(m - m2), p = expf(d - m2);
        l = l * f + p;
        for (int c = 0; c < 4; ++c) acc[c] = acc[c] * f + p * to_f32(v[c * 32 + lane]);
        m = m2;
    }
    for (int c = 0; c < 4; ++c)
        a.out[((size_t)tok * a.H + h) * kHeadDim + c * 32 + lane] = __float2bfloat16_rn(l > 0.f ? acc[c] / l : 0.f);
    if (lane == 0) a.lse[tok * a.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

bool al(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace

kda_status_t check_latent(const void *q, const void *k, const void *v, const void *k_shared, const int32_t *cu_q,
                          const int32_t *cu_k, const void *out, const float *lse, int B, int T, int Tk, int H, int N,
                          int dk, int dv, int dr, long long k_tok, long long k_head, long long v_tok, long long v_head,
                          long long r_tok, float scale, kda_dtype_t dtype, const void *workspace, size_t workspace_bytes,
                          size_t need, LatentArgs *a)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || Tk < 0 || N < 0 || H <= 0) return KDA_ERR_INVALID_ARG;
    if ((cu_q == nullptr) != (cu_k == nullptr)) return KDA_ERR_INVALID_ARG;
    if (cu_q ? (B != 1 || !al(cu_q, 4) || !al(cu_k, 4)) : N != B) return KDA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (!workspace || !al(workspace, 16) || need == 0 || workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 || dk != kHeadDim || dv != kHeadDim || (dr != 0 && dr != kSharedDim)) return KDA_ERR_UNSUPPORTED;
    if (H > kMaxGridDim || N > kMaxGridDim) return KDA_ERR_UNSUPPORTED;
    if ((long long)B * T > 0x7fffffffLL || (long long)B * Tk > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if ((long long)B * T > 0 && (!q || !out || !lse)) return KDA_ERR_INVALID_ARG;
    if ((long long)B * Tk > 0 && (!k || !v || (dr && !k_shared))) return KDA_ERR_INVALID_ARG;
    if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(k_shared, 16) || !al(out, 16) || !al(lse, 4)) return KDA_ERR_INVALID_ARG;
    if (k_tok % 8 || k_head % 8 || v_tok % 8 || v_head % 8 || (dr && r_tok % 8)) return KDA_ERR_INVALID_ARG;
    if (k_tok <= 0 || k_head <= 0 || v_tok <= 0 || v_head <= 0 || (dr && r_tok <= 0)) return KDA_ERR_INVALID_ARG;
    a->q = (const __nv_bfloat16 *)q; a->k = (const __nv_bfloat16 *)k; a->v = (const __nv_bfloat16 *)v;
    a->r = dr ? (const __nv_bfloat16 *)k_shared : nullptr;
    a->k_tok = k_tok; a->k_head = k_head; a->v_tok = v_tok; a->v_head = v_head; a->r_tok = r_tok;
    a->cu_q = cu_q; a->cu_k = cu_k; a->out = (__nv_bfloat16 *)out; a->lse = const_cast<float *>(lse);
    a->B = B; a->T = T; a->Tk = Tk; a->H = H; a->N = N; a->R = dr; a->scale = scale;
    a->status = (int32_t *)workspace;
    return KDA_OK;
}

cudaError_t launch_latent_fwd(const LatentArgs &a, cudaStream_t stream)
{
    const long long tokens = (long long)a.B * a.T;
    latent_fwd_simple<<<dim3((unsigned)((tokens + 3) / 4), a.H), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_latent_fwd_workspace_size(int B, int T, int Tk, int H, int N, int dr)
{
    if (B < 0 || T < 0 || Tk < 0 || H <= 0 || N < 0 || (dr != 0 && dr != kSharedDim)) return 0;
    return kStatusBytes;
}

kda_status_t kda_latent_fwd(const void *q, const void *k, const void *v, const void *k_shared, const int32_t *cu_seqlens,
                            const int32_t *cu_seqlens_k, void *out, float *lse, int B, int T, int Tk, int H, int N, int dk,
                            int dv, int dr, long long k_token_stride, long long k_head_stride, long long v_token_stride,
                            long long v_head_stride, long long shared_token_stride, int causal, float scale,
                            kda_dtype_t dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    LatentArgs a;
    const kda_status_t s = check_latent(q, k, v, k_shared, cu_seqlens, cu_seqlens_k, out, lse, B, T, Tk, H, N, dk, dv, dr,
                                        k_token_stride, k_head_stride, v_token_stride, v_head_stride, shared_token_stride,
                                        scale, dtype, workspace, workspace_bytes,
                                        kda_latent_fwd_workspace_size(B, T, Tk, H, N, dr), &a);
    if (s != KDA_OK) return s;
    a.causal = causal != 0;
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemsetAsync(workspace, 0, kStatusBytes, st) != cudaSuccess) return KDA_ERR_CUDA;
    if ((long long)B * T == 0 || N == 0) return KDA_OK;
    return launch_latent_fwd(a, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
