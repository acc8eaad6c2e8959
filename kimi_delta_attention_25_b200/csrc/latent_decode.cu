// latent_decode.cu -- the absorbed form of the latent attention, for one or a few new tokens per sequence
// over a paged cache. Cache row j holds the token's latent vector c_j (512) and its shared key part r_j (64,
// or none); every head reads the same rows, as keys and (the latent) as values:
//   s_j = scale (q[:512] . c_j + q[512:] . r_j),   o = sum_j softmax_j(s) c_j   (512 values per head).
// Token t of a sequence's Tq new ones (the last of its seq_len cached tokens) sees the rows up to its own.
#include "kda_internal.cuh"

namespace kda {
namespace {

struct DecodeArgs {
    const __nv_bfloat16 *q, *cache;
    const int32_t *table, *lens;
    __nv_bfloat16 *out;
    float *lse;
    int N, Tq, H, R, page, pages, max_pages;
    float scale;
    int32_t *status;
};

// One warp per (sequence, token, head).
__global__ void __launch_bounds__(128) latent_decode_simple(DecodeArgs a)
{
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)a.N * a.Tq * a.H) return;
    const int n = (int)(row / ((long long)a.Tq * a.H)), t = (int)(row / a.H % a.Tq), W = kLatentDim + a.R;
    long long len = a.lens[n];
    if (len < 0 || len > (long long)a.max_pages * a.page) { set_status(a.status, KDA_ERR_INVALID_ARG); len = 0; }
    float q[18], acc[16] = {}, m = -INFINITY, l = 0.f;
    for (int c = 0; c < W / 32; ++c) q[c] = to_f32(a.q[row * W + c * 32 + lane]);
    for (long long j = 0; j < len - a.Tq + t + 1; ++j) {
        const int pg = a.table[(size_t)n * a.max_pages + j / a.page];
        if (pg < 0 || pg >= a.pages) { set_status(a.status, KDA_ERR_INVALID_ARG); continue; }
        const __nv_bfloat16 *c = a.cache + ((size_t)pg * a.page + j % a.page) * W;
        float x[18], d = 0.f;
        for (int i = 0; i < W / 32; ++i) { x[i] = to_f32(c[i * 32 + lane]); d += q[i] * x[i]; }
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        d *= a.scale;
        const float m2 = fmaxf(m, d);
        if (m2 == -INFINITY) continue;
        const float f = expf(m - m2), p = expf(d - m2);
        l = l * f + p;
        for (int i = 0; i < 16; ++i) acc[i] = acc[i] * f + p * x[i];
        m = m2;
    }
    for (int i = 0; i < 16; ++i) a.out[row * kLatentDim + i * 32 + lane] = __float2bfloat16_rn(l > 0.f ? acc[i] / l : 0.f);
    if (lane == 0) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

bool al(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_latent_decode_workspace_size(int N, int Tq, int H)
{
    if (N < 0 || Tq < 1 || H < 1) return 0;
    return kStatusBytes;
}

kda_status_t kda_latent_decode_step(const void *q, const void *cache, const int32_t *page_table, const int32_t *seq_lens,
                                    void *out, float *lse, int N, int Tq, int H, int dc, int dr, int page_size,
                                    long long num_pages, int max_pages, float scale, kda_dtype_t dtype, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (N < 0 || Tq < 1 || H < 1 || page_size < 1 || num_pages < 0 || max_pages < 0) return KDA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (!workspace || !al(workspace, 16) || workspace_bytes < kda_latent_decode_workspace_size(N, Tq, H)) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 || dc != kLatentDim || (dr != 0 && dr != kSharedDim) || page_size % 16 != 0) return KDA_ERR_UNSUPPORTED;
    if (num_pages * page_size > 0x7fffffffLL || (long long)max_pages * page_size > 0x7fffffffLL ||
        (long long)N * Tq * H > 0x7fffffffLL || N > kMaxGridDim)
        return KDA_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    if (N > 0) {
        if (!q || !seq_lens || !out || !lse) return KDA_ERR_INVALID_ARG;
        if (!al(q, 16) || !al(cache, 16) || !al(page_table, 4) || !al(seq_lens, 4) || !al(out, 16) || !al(lse, 4))
            return KDA_ERR_INVALID_ARG;
        if (max_pages > 0 && (!page_table || (num_pages > 0 && !cache))) return KDA_ERR_INVALID_ARG;
    }
    if (cudaMemsetAsync(workspace, 0, kStatusBytes, st) != cudaSuccess) return KDA_ERR_CUDA;
    if (N == 0) return KDA_OK;
    DecodeArgs a;
    a.q = (const __nv_bfloat16 *)q; a.cache = (const __nv_bfloat16 *)cache; a.table = page_table; a.lens = seq_lens;
    a.out = (__nv_bfloat16 *)out; a.lse = lse; a.N = N; a.Tq = Tq; a.H = H; a.R = dr; a.page = page_size;
    a.pages = (int)num_pages; a.max_pages = max_pages; a.scale = scale; a.status = (int32_t *)workspace;
    const long long rows = (long long)N * Tq * H;
    latent_decode_simple<<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
