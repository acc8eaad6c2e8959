// latent_bwd.cu -- the backward pass of the expanded latent attention (latent_fwd.cu), with P recomputed
// from the forward's lse:  P = exp(s - lse),  D_i = do_i . o_i,  dP = do v^T,  dS = P (dP - D),
//   dq = scale dS [k, r],  dk = scale dS^T q[:128],  dr = scale sum_h dS^T q[128:],  dv = P^T do.
#include "latent.cuh"

namespace kda {
namespace {

// D_i = do_i . o_i, one warp per (token, head).
__global__ void __launch_bounds__(256) latent_delta_kernel(const __nv_bfloat16 *__restrict__ out, const __nv_bfloat16 *__restrict__ dout,
                                                           float *__restrict__ delta, long long rows)
{
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const uint2 o = reinterpret_cast<const uint2 *>(out + row * kHeadDim)[lane], d = reinterpret_cast<const uint2 *>(dout + row * kHeadDim)[lane];
    float s = __uint_as_float(o.x << 16) * __uint_as_float(d.x << 16);
    s += __uint_as_float(o.x & 0xFFFF0000u) * __uint_as_float(d.x & 0xFFFF0000u);
    s += __uint_as_float(o.y << 16) * __uint_as_float(d.y << 16);
    s += __uint_as_float(o.y & 0xFFFF0000u) * __uint_as_float(d.y & 0xFFFF0000u);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lane == 0) delta[row] = s;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// One warp per (query, head): dq.
__global__ void __launch_bounds__(128) latent_dq_simple(LatentArgs a, LatentBwdArgs b)
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
    float qv[6] = {}, dov[4], acc[6] = {};
    for (int c = 0; c < W / 32; ++c) qv[c] = to_f32(a.q[((size_t)tok * a.H + h) * W + c * 32 + lane]);
    for (int c = 0; c < 4; ++c) dov[c] = to_f32(b.dout[((size_t)tok * a.H + h) * kHeadDim + c * 32 + lane]);
    const float lse = a.lse[tok * a.H + h], delta = b.delta[tok * a.H + h];
    const long long hi = a.causal ? min(s.k1 - s.k0, tok - s.q0 + (s.k1 - s.k0) - (s.q1 - s.q0) + 1) : s.k1 - s.k0;
    for (long long j = 0; j < hi; ++j) {
        const __nv_bfloat16 *k = a.k + (s.k0 + j) * a.k_tok + h * a.k_head, *v = a.v + (s.k0 + j) * a.v_tok + h * a.v_head;
        const __nv_bfloat16 *r = a.r + (s.k0 + j) * a.r_tok;
        float d = 0.f, dp = 0.f;
        for (int c = 0; c < 4; ++c) { d += qv[c] * to_f32(k[c * 32 + lane]); dp += dov[c] * to_f32(v[c * 32 + lane]); }
        if (a.R) for (int c = 0; c < 2; ++c) d += qv[4 + c] * to_f32(r[c * 32 + lane]);
        d = warp_sum(d) * a.scale;
        dp = warp_sum(dp);
        const float ds = (lse == -INFINITY ? 0.f : expf(d - lse)) * (dp - delta) * a.scale;
        for (int c = 0; c < 4; ++c) acc[c] += ds * to_f32(k[c * 32 + lane]);
        if (a.R) for (int c = 0; c < 2; ++c) acc[4 + c] += ds * to_f32(r[c * 32 + lane]);
    }
    for (int c = 0; c < W / 32; ++c) b.dq[((size_t)tok * a.H + h) * W + c * 32 + lane] = __float2bfloat16_rn(acc[c]);
}

// One warp per (key, head): dk, dv and the head's part of dr.
__global__ void __launch_bounds__(128) latent_dkv_simple(LatentArgs a, LatentBwdArgs b)
{
    const long long key = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = blockIdx.y, lane = threadIdx.x & 31;
    if (key >= (long long)a.B * a.Tk) return;
    const int n = latent_sequence(a.cu_k, a.N, a.Tk, key);
    LatentSpan s;
    if (n < 0 || !latent_span(a.cu_q, a.cu_k, n, a.T, a.Tk, &s)) return;
    const int W = kHeadDim + a.R;
    float kv[6] = {}, vv[4], dk[6] = {}, dv[4] = {};
    for (int c = 0; c < 4; ++c) {
        kv[c] = to_f32(a.k[key * a.k_tok + h * a.k_head + c * 32 + lane]);
        vv[c] = to_f32(a.v[key * a.v_tok + h * a.v_head + c * 32 + lane]);
    }
    if (a.R) for (int c = 0; c < 2; ++c) kv[4 + c] = to_f32(a.r[key * a.r_tok + c * 32 + lane]);
    long long lo = a.causal ? (key - s.k0) - (s.k1 - s.k0) + (s.q1 - s.q0) : 0;
    if (lo < 0) lo = 0;
    for (long long tok = s.q0 + lo; tok < s.q1; ++tok) {
        const __nv_bfloat16 *q = a.q + ((size_t)tok * a.H + h) * W, *dout = b.dout + ((size_t)tok * a.H + h) * kHeadDim;
        float qv[6] = {}, dov[4], d = 0.f, dp = 0.f;
        for (int c = 0; c < W / 32; ++c) { qv[c] = to_f32(q[c * 32 + lane]); d += qv[c] * kv[c]; }
        for (int c = 0; c < 4; ++c) { dov[c] = to_f32(dout[c * 32 + lane]); dp += dov[c] * vv[c]; }
        d = warp_sum(d) * a.scale;
        dp = warp_sum(dp);
        const float lse = a.lse[tok * a.H + h], p = lse == -INFINITY ? 0.f : expf(d - lse);
        const float ds = p * (dp - b.delta[tok * a.H + h]) * a.scale;
        for (int c = 0; c < W / 32; ++c) dk[c] += ds * qv[c];
        for (int c = 0; c < 4; ++c) dv[c] += p * dov[c];
    }
    for (int c = 0; c < 4; ++c) {
        b.dk[((size_t)key * a.H + h) * kHeadDim + c * 32 + lane] = __float2bfloat16_rn(dk[c]);
        b.dv[((size_t)key * a.H + h) * kHeadDim + c * 32 + lane] = __float2bfloat16_rn(dv[c]);
    }
    if (a.R) for (int c = 0; c < 2; ++c) b.dr_head[((size_t)key * a.H + h) * kSharedDim + c * 32 + lane] = dk[4 + c];
}

// dr[key] = sum over heads of dr_head[key][h], in fp32 and in head order. 16 keys per block: 16 threads of a
// float4 each per key.
__global__ void __launch_bounds__(256) latent_dr_kernel(const float *__restrict__ dr_head, __nv_bfloat16 *__restrict__ dr, long long keys, int H)
{
    const long long key = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int c = (threadIdx.x & 15) * 4;
    if (key >= keys) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int h = 0; h < H; ++h) {
        const float4 x = *reinterpret_cast<const float4 *>(dr_head + ((size_t)key * H + h) * kSharedDim + c);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    uint2 u = make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
    *reinterpret_cast<uint2 *>(dr + (size_t)key * kSharedDim + c) = u;
}

bool al(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace

cudaError_t launch_latent_bwd(const LatentArgs &a, const LatentBwdArgs &b, cudaStream_t stream)
{
    const long long tokens = (long long)a.B * a.T, keys = (long long)a.B * a.Tk, rows = tokens * a.H;
    if (tokens > 0) {
        latent_delta_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(a.out, b.dout, b.delta, rows);
        latent_dq_simple<<<dim3((unsigned)((tokens + 3) / 4), a.H), 128, 0, stream>>>(a, b);
    }
    if (keys > 0) {
        latent_dkv_simple<<<dim3((unsigned)((keys + 3) / 4), a.H), 128, 0, stream>>>(a, b);
        if (a.R) latent_dr_kernel<<<(unsigned)((keys + 15) / 16), 256, 0, stream>>>(b.dr_head, b.dr, keys, a.H);
    }
    return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

namespace {
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
}

extern "C" {

size_t kda_latent_bwd_workspace_size(int B, int T, int Tk, int H, int N, int dr)
{
    if (B < 0 || T < 0 || Tk < 0 || H <= 0 || N < 0 || (dr != 0 && dr != kSharedDim)) return 0;
    return kStatusBytes + align256((size_t)B * T * H * 4) + align256((size_t)B * Tk * H * dr * 4);
}

kda_status_t kda_latent_bwd(const void *q, const void *k, const void *v, const void *k_shared, const int32_t *cu_seqlens,
                            const int32_t *cu_seqlens_k, const void *out, const float *lse, const void *dout, void *dq,
                            void *dk_out, void *dv_out, void *dk_shared, int B, int T, int Tk, int H, int N, int dk, int dv,
                            int dr, long long k_token_stride, long long k_head_stride, long long v_token_stride,
                            long long v_head_stride, long long shared_token_stride, int causal, float scale,
                            kda_dtype_t dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    LatentArgs a;
    const kda_status_t s = check_latent(q, k, v, k_shared, cu_seqlens, cu_seqlens_k, out, lse, B, T, Tk, H, N, dk, dv, dr,
                                        k_token_stride, k_head_stride, v_token_stride, v_head_stride, shared_token_stride,
                                        scale, dtype, workspace, workspace_bytes,
                                        kda_latent_bwd_workspace_size(B, T, Tk, H, N, dr), &a);
    if (s != KDA_OK) return s;
    if ((long long)B * T > 0 && (!dout || !dq)) return KDA_ERR_INVALID_ARG;
    if ((long long)B * Tk > 0 && (!dk_out || !dv_out || (dr && !dk_shared))) return KDA_ERR_INVALID_ARG;
    if (!al(dout, 16) || !al(dq, 16) || !al(dk_out, 16) || !al(dv_out, 16) || !al(dk_shared, 16)) return KDA_ERR_INVALID_ARG;
    a.causal = causal != 0;
    LatentBwdArgs b;
    b.dout = (const __nv_bfloat16 *)dout;
    b.dq = (__nv_bfloat16 *)dq; b.dk = (__nv_bfloat16 *)dk_out; b.dv = (__nv_bfloat16 *)dv_out; b.dr = (__nv_bfloat16 *)dk_shared;
    b.delta = (float *)((unsigned char *)workspace + kStatusBytes);
    b.dr_head = (float *)((unsigned char *)b.delta + align256((size_t)B * T * H * 4));
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemsetAsync(workspace, 0, kStatusBytes, st) != cudaSuccess) return KDA_ERR_CUDA;
    if (N == 0 || B == 0) return KDA_OK;
    return launch_latent_bwd(a, b, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
