// rms_norm.cu -- the root-mean-square norm in front of a layer (with the residual's addition, and
// with an 8-bit output for 8-bit projections), its backward pass, and the cache append of the
// latent attention (the latent's norm and the shared key part, written into cache rows).
//
//   h = x + residual (rounded to the type, kept),  r = 1 / sqrt(mean_c h_c^2 + eps),  y = h r w
//   8 bits: over each group of 128 channels  s = max |y| / 448,  q = y / s in e4m3 (448: its largest)
//   backward: g = w dy,  dx = r (g - h r^2 mean_c(g h)) + dh,  dw = sum over rows of dy h r
//
// All of them are bound by memory: each input is read once and each output written once, a few flops
// per element. A row is held in registers between the sum of squares and the scaling, by TPR threads
// of at most VPT 16-byte vectors each; TPR is the smallest of 32, 128 and 512 that holds the row, so
// that short rows need no block barrier and long ones stay in registers. Sums are fp32.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kda_internal.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

constexpr int kNormMaxWidth = 16384;
constexpr int kGroup = 128;              // channels that share one scale of the 8-bit output
constexpr float kE4m3Max = 448.f;

// A 16-byte vector of T as floats: 8 bf16 or 4 fp32.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = __uint_as_float(w[i] << 16); f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u); }
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f[2 * i])) |
                   ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f[2 * i + 1])) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *red)
{
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int w = 1; w < TPR / 32; ++w) x += red[w];
    }
    return x;
}

struct NormParams {
    const void *x, *res;
    const float *w;
    void *y, *h;          // y: dtype or e4m3; h: dtype, null without a residual
    float *scale;         // 8-bit output: [rows, D / 128]
    float eps, inv_d;
    long long rows;
    int D;
};

// TPR threads per row, block of max(TPR, 128) threads (four rows of a warp each when TPR = 32).
template <typename T, int TPR, int VPT, bool RES, bool Q8>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128) rms_norm_kernel(NormParams p)
{
    constexpr int NV = Vec<T>::n;
    __shared__ float red[TPR / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
    if (row >= p.rows) return;               // whole warps (TPR 32), or never (one row per block)
    const int nvec = p.D / NV;
    const size_t base = (size_t)row * nvec;
    uint4 xv[VPT], rv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * TPR + t;
        xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
        if (v < nvec) {
            xv[i] = __ldcs((const uint4 *)p.x + base + v);
            if constexpr (RES) rv[i] = __ldcs((const uint4 *)p.res + base + v);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float f[NV];
        Vec<T>::unpack(xv[i], f);
        if constexpr (RES) {
            float g[NV];
            Vec<T>::unpack(rv[i], g);
#pragma unroll
            for (int e = 0; e < NV; ++e) f[e] += g[e];
            xv[i] = Vec<T>::pack(f);          // the sum as it is kept: what is normalised, and read back by the backward pass
            const int v = i * TPR + t;
            if (v < nvec) ((uint4 *)p.h)[base + v] = xv[i];
            Vec<T>::unpack(xv[i], f);
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) ss += f[e] * f[e];
    }
    ss = row_sum<TPR>(ss, red);
    const float r = 1.f / sqrtf(ss * p.inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * TPR + t;
        float f[NV], y[NV];
        Vec<T>::unpack(xv[i], f);
#pragma unroll
        for (int e = 0; e < NV; e += 4) {
            const float4 w = v < nvec ? *reinterpret_cast<const float4 *>(p.w + (size_t)v * NV + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            y[e] = f[e] * r * w.x; y[e + 1] = f[e + 1] * r * w.y; y[e + 2] = f[e + 2] * r * w.z; y[e + 3] = f[e + 3] * r * w.w;
        }
        if constexpr (!Q8) {
            if (v < nvec) ((uint4 *)p.y)[base + v] = Vec<T>::pack(y);
        } else {
            // a group is 128 / NV consecutive lanes (16 or 32); lanes behind the row's end hold zeros
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < NV; ++e) m = fmaxf(m, fabsf(y[e]));
            bool nan = false;
#pragma unroll
            for (int e = 0; e < NV; ++e) nan |= y[e] != y[e];
            if (nan) m = __int_as_float(0x7fc00000);
#pragma unroll
            for (int o = kGroup / NV / 2; o > 0; o >>= 1) {
                const float other = __shfl_xor_sync(0xffffffffu, m, o);
                m = (m != m) ? m : (other != other ? other : fmaxf(m, other));
            }
            const float s = m / kE4m3Max;
            const float d = s == 0.f ? 1.f : s;
            if (v < nvec) {
                uint16_t q[NV / 2];
#pragma unroll
                for (int e = 0; e < NV; e += 2)
                    q[e / 2] = __nv_cvt_float2_to_fp8x2(make_float2(y[e] / d, y[e + 1] / d), __NV_SATFINITE, __NV_E4M3);
                if constexpr (NV == 8) {
                    reinterpret_cast<uint2 *>(p.y)[base + v] =
                        make_uint2(q[0] | ((uint32_t)q[1] << 16), q[2] | ((uint32_t)q[3] << 16));
                } else {
                    reinterpret_cast<uint32_t *>(p.y)[base + v] = q[0] | ((uint32_t)q[1] << 16);
                }
                if (v % (kGroup / NV) == 0) p.scale[(size_t)row * (p.D / kGroup) + v / (kGroup / NV)] = s;
            }
        }
    }
}

struct NormBwdParams {
    const void *dy, *h, *dh;
    const float *w;
    void *dx;
    float *partial;       // [gridDim.x, D]: each block's sum of dy h r
    float eps, inv_d;
    long long rows;
    int D;
};

__device__ __forceinline__ void bulk_row(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(sm100::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(sm100::smem_u32(bar)) : "memory");
}

// TPR threads hold one row, and the block walks its rows with the weight gradient's sum in registers;
// a second kernel adds the blocks' sums in a fixed order, so results do not depend on timing. Up to 1024 vectors
// a row (one a thread) the rows come through shared memory, kRowsAhead of them by bulk copies of one thread, which
// keeps 190 KB an SM on their way without a register (8192 x 4096 bf16, both kernels: rows loaded into registers one
// ahead took 67 us, this 50 to 52); wider rows are loaded as they are needed.
constexpr int kRowsAhead = 4;
template <typename T, int TPR, int VPT, bool DH>
__global__ void __launch_bounds__(TPR) rms_norm_bwd_kernel(NormBwdParams p)
{
    constexpr int NV = Vec<T>::n;
    constexpr bool AHEAD = VPT == 1;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][TPR / 32][2];
    __shared__ uint64_t full[kRowsAhead];
    __shared__ int stop;                     // a wait ran out (1), and the copies in flight have been waited for (2)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x, nvec = p.D / NV;
    const uint32_t row_bytes = (uint32_t)nvec * 16;
    float dw[VPT][NV], w1[AHEAD ? NV : 1];
    auto weights = [&](int v, float *w) {
#pragma unroll
        for (int e = 0; e < NV; e += 4) {
            const float4 w4 = v < nvec ? *reinterpret_cast<const float4 *>(p.w + (size_t)v * NV + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            w[e] = w4.x; w[e + 1] = w4.y; w[e + 2] = w4.z; w[e + 3] = w4.w;
        }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < NV; ++e) dw[i][e] = 0.f;
    auto fetch = [&](const void *src, long long row, int v) {
        return v < nvec ? __ldcs((const uint4 *)src + (size_t)row * nvec + v) : make_uint4(0, 0, 0, 0);
    };
    auto order = [&](long long row, int s) {                  // one thread: the row's tensors into stage s
        if (row >= p.rows) return;
        unsigned char *dst = ring + (size_t)s * (DH ? 3 : 2) * row_bytes;
        sm100::mbar_arrive_expect_tx(&full[s], (DH ? 3 : 2) * row_bytes);
        bulk_row(dst, (const unsigned char *)p.h + (size_t)row * row_bytes, row_bytes, &full[s]);
        bulk_row(dst + row_bytes, (const unsigned char *)p.dy + (size_t)row * row_bytes, row_bytes, &full[s]);
        if constexpr (DH) bulk_row(dst + 2 * row_bytes, (const unsigned char *)p.dh + (size_t)row * row_bytes, row_bytes, &full[s]);
    };
    if constexpr (AHEAD) {
        if (t == 0) {
            for (int s = 0; s < kRowsAhead; ++s) sm100::mbar_init(&full[s], 1);
            stop = 0;
            sm100::fence_mbar_init();
        }
        __syncthreads();
        if (t == 0)
            for (int s = 0; s < kRowsAhead; ++s) order(blockIdx.x + (long long)s * gridDim.x, s);
        weights(t, w1);
    }
    // A wait that runs out (the call has no status word to record it in): from that row on this thread's sum is NaN, and with
    // it the block's rows of dx and all of dweight. The other waits then give up at once, no copy is ordered any more, and
    // what is in flight lands before the block ends.
    bool stopped = false;
    auto arrived = [&](int s, uint32_t parity) {
        if (sm100::mbar_try_wait(&full[s], parity)) return true;
        const long long t0 = clock64();
        while (!sm100::mbar_try_wait(&full[s], parity)) {
            if (*(volatile int *)&stop) return false;
            if (clock64() - t0 > 4000000000LL) { *(volatile int *)&stop = 1; return false; }
        }
        return true;
    };
    int it = 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
        const int flip = it & 1, stage = it % kRowsAhead;
        uint4 hv[VPT], gv[VPT], ev = make_uint4(0, 0, 0, 0);
        if constexpr (AHEAD) {
            stopped = stopped || !arrived(stage, (it / kRowsAhead) & 1);
            const uint4 *src = reinterpret_cast<const uint4 *>(ring + (size_t)stage * (DH ? 3 : 2) * row_bytes);
            hv[0] = gv[0] = make_uint4(0, 0, 0, 0);
            if (t < nvec) {
                hv[0] = src[t];
                gv[0] = src[nvec + t];
                if constexpr (DH) ev = src[2 * nvec + t];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) { hv[i] = fetch(p.h, row, i * TPR + t); gv[i] = fetch(p.dy, row, i * TPR + t); }
        }
        float ss = AHEAD && stopped ? __int_as_float(0x7fc00000) : 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float h[NV], g[NV], wl[NV];
            Vec<T>::unpack(hv[i], h);
            Vec<T>::unpack(gv[i], g);
            if constexpr (!AHEAD) weights(i * TPR + t, wl);
            const float *w = AHEAD ? w1 : wl;
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                ss += h[e] * h[e];
                sg += g[e] * w[e] * h[e];
            }
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, m);
            sg += __shfl_xor_sync(0xffffffffu, sg, m);
        }
        // two buffers in turn: one barrier a row is enough; behind it every thread has read the row's stage
        if constexpr (TPR > 32) {
            if ((t & 31) == 0) { red[flip][t >> 5][0] = ss; red[flip][t >> 5][1] = sg; }
            __syncthreads();
        } else {
            __syncwarp();
        }
        if constexpr (AHEAD)
            if (t == 0) {
                if (!stopped) order(row + (long long)kRowsAhead * gridDim.x, stage);
                else if (*(volatile int *)&stop != 2) {
                    for (int i = it; i < it + kRowsAhead; ++i)
                        (void)sm100::mbar_wait(&full[i % kRowsAhead], (i / kRowsAhead) & 1, 100000000LL);
                    *(volatile int *)&stop = 2;
                }
            }
        if constexpr (TPR > 32) {
            ss = red[flip][0][0];
            sg = red[flip][0][1];
#pragma unroll
            for (int x = 1; x < TPR / 32; ++x) { ss += red[flip][x][0]; sg += red[flip][x][1]; }
        }
        const float r = 1.f / sqrtf(ss * p.inv_d + p.eps), c = r * r * (sg * p.inv_d);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * TPR + t;
            float h[NV], g[NV], d[NV], wl[NV];
            Vec<T>::unpack(hv[i], h);
            Vec<T>::unpack(gv[i], g);
            if constexpr (DH && !AHEAD) ev = fetch(p.dh, row, v);
            Vec<T>::unpack(ev, d);
            if constexpr (!AHEAD) weights(v, wl);
            const float *w = AHEAD ? w1 : wl;
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                dw[i][e] += g[e] * (h[e] * r);
                d[e] += r * (g[e] * w[e] - h[e] * c);
            }
            if (v < nvec) ((uint4 *)p.dx)[(size_t)row * nvec + v] = Vec<T>::pack(d);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * TPR + t;
        if (v < nvec) {
#pragma unroll
            for (int e = 0; e < NV; e += 4)
                *reinterpret_cast<float4 *>(p.partial + (size_t)blockIdx.x * p.D + (size_t)v * NV + e) =
                    make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
        }
    }
}

// dw[c] = sum over blocks of partial[block][c]: 32 channels per CTA, 32 warps over the blocks.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float *__restrict__ partial, float *__restrict__ dw,
                                                           int blocks, int D)
{
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float a = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c < D) {
#pragma unroll 16
        for (int b = warp; b < blocks; b += 32) a += partial[(size_t)b * D + c];
    }
    s[warp][lane] = a;
    __syncthreads();
    a = s[lane][warp];                        // channel `warp` of the CTA, over the 32 sums
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
    if (lane == 0 && blockIdx.x * 32 + warp < D) dw[blockIdx.x * 32 + warp] = a;
}

// One warp per token: 16 of the 512 latent channels per lane (two vectors), then the shared key part.
__global__ void __launch_bounds__(128) latent_append_kernel(const __nv_bfloat16 *__restrict__ c, const __nv_bfloat16 *__restrict__ k_shared,
                                                            const long long *__restrict__ slots, const float *__restrict__ w,
                                                            __nv_bfloat16 *__restrict__ cache, long long c_stride,
                                                            long long r_stride, long long cache_rows, int T, int R, float eps)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    const long long slot = slots[t];
    if (slot < 0 || slot >= cache_rows) return;
    using V = Vec<__nv_bfloat16>;
    const uint4 *src = (const uint4 *)(c + (size_t)t * c_stride);
    uint4 *dst = (uint4 *)(cache + (size_t)slot * (kLatentDim + R));
    uint4 a[2] = {src[lane], src[32 + lane]};
    uint4 rv = make_uint4(0, 0, 0, 0);
    const bool tail = lane < R / 8;
    if (tail) rv = ((const uint4 *)(k_shared + (size_t)t * r_stride))[lane];
    if (w) {
        float f[2][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            V::unpack(a[i], f[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += f[i][e] * f[i][e];
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = 1.f / sqrtf(ss * (1.f / kLatentDim) + eps);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 wv = *reinterpret_cast<const float4 *>(w + (i * 32 + lane) * 8 + e);
                f[i][e] *= r * wv.x; f[i][e + 1] *= r * wv.y; f[i][e + 2] *= r * wv.z; f[i][e + 3] *= r * wv.w;
            }
            a[i] = V::pack(f[i]);
        }
    }
    dst[lane] = a[0];
    dst[32 + lane] = a[1];
    if (tail) dst[64 + lane] = rv;
}

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <typename T, bool RES, bool Q8>
cudaError_t launch_norm(const NormParams &p, cudaStream_t st)
{
    const int nvec = p.D / Vec<T>::n;
    auto go = [&](auto kern, int tpr) {
        const int threads = tpr > 128 ? tpr : 128, per = threads / tpr;
        return launch_after(kern, (unsigned)((p.rows + per - 1) / per), threads, 0, st, p);
    };
    if (nvec <= 32 * 4) return go(rms_norm_kernel<T, 32, 4, RES, Q8>, 32);
    if (nvec <= 128 * 4) return go(rms_norm_kernel<T, 128, 4, RES, Q8>, 128);
    if (nvec <= 512 * 4) return go(rms_norm_kernel<T, 512, 4, RES, Q8>, 512);
    return go(rms_norm_kernel<T, 512, 8, RES, Q8>, 512);
}

kda_status_t run_norm(const void *x, const void *residual, const float *weight, void *y, float *scale, void *h,
                      long long rows, int D, float eps, kda_dtype_t dtype, bool q8, void *stream)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (rows < 0 || D <= 0 || !(eps >= 0.f) || eps > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > kNormMaxWidth || (q8 && D % kGroup != 0) || rows > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!x || !weight || !y || (q8 && !scale) || (residual && !h)) return KDA_ERR_INVALID_ARG;
    if (!al(x, 16) || !al(residual, 16) || !al(weight, 16) || !al(y, 16) || !al(h, 16) || !al(scale, 4))
        return KDA_ERR_INVALID_ARG;
    if (q8) {
        // rows of y have other places than those of x: another block would write over what one has yet to read
        const uintptr_t y0 = (uintptr_t)y, y1 = y0 + (size_t)rows * D, wide = (size_t)rows * D * (dtype == KDA_BF16 ? 2 : 4);
        for (const void *t : {x, residual, (const void *)h})
            if (t && y0 < (uintptr_t)t + wide && (uintptr_t)t < y1) return KDA_ERR_INVALID_ARG;
    }
    NormParams p;
    p.x = x; p.res = residual; p.w = weight; p.y = y; p.h = h; p.scale = scale; p.eps = eps; p.inv_d = 1.f / (float)D;
    p.rows = rows; p.D = D;
    cudaStream_t st = (cudaStream_t)stream;
    using bf = __nv_bfloat16;
    cudaError_t e;
    if (dtype == KDA_BF16) {
        if (residual) e = q8 ? launch_norm<bf, true, true>(p, st) : launch_norm<bf, true, false>(p, st);
        else e = q8 ? launch_norm<bf, false, true>(p, st) : launch_norm<bf, false, false>(p, st);
    } else {
        if (residual) e = q8 ? launch_norm<float, true, true>(p, st) : launch_norm<float, true, false>(p, st);
        else e = q8 ? launch_norm<float, false, true>(p, st) : launch_norm<float, false, false>(p, st);
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Threads that hold a row of the backward pass, and its blocks: 1024 threads on each of 148 SMs.
int bwd_threads(int nvec)
{
    return nvec <= 32 ? 32 : nvec <= 128 ? 128 : nvec <= 256 ? 256 : nvec <= 512 ? 512 : nvec <= 1024 ? 1024 : 512;
}
int bwd_blocks(long long rows, int nvec)
{
    const long long most = 148 * 1024 / bwd_threads(nvec);
    return (int)(rows < most ? (rows > 0 ? rows : 1) : most);
}

template <typename T, bool DH>
cudaError_t launch_norm_bwd(const NormBwdParams &p, int blocks, cudaStream_t st)
{
    const int nvec = p.D / Vec<T>::n;
    const int ring = nvec <= 1024 ? kRowsAhead * (DH ? 3 : 2) * nvec * 16 : 0;
    auto go = [&](auto kern, int threads) {
        if (ring > 32 * 1024) {               // (48 KB, the static part among them, need no leave)
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
            if (e != cudaSuccess) return e;
        }
        return launch_after(kern, blocks, threads, ring, st, p);
    };
    if (nvec <= 32) return go(rms_norm_bwd_kernel<T, 32, 1, DH>, 32);
    if (nvec <= 128) return go(rms_norm_bwd_kernel<T, 128, 1, DH>, 128);
    if (nvec <= 256) return go(rms_norm_bwd_kernel<T, 256, 1, DH>, 256);
    if (nvec <= 512) return go(rms_norm_bwd_kernel<T, 512, 1, DH>, 512);
    if (nvec <= 1024) return go(rms_norm_bwd_kernel<T, 1024, 1, DH>, 1024);
    if constexpr (Vec<T>::n == 4)
        if (nvec > 512 * 4) return go(rms_norm_bwd_kernel<T, 512, 8, DH>, 512);
    return go(rms_norm_bwd_kernel<T, 512, 4, DH>, 512);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_rms_norm(const void *x, const void *residual, const float *weight, void *y, void *h, long long rows,
                          int D, float eps, kda_dtype_t dtype, void *stream)
{
    return run_norm(x, residual, weight, y, nullptr, h, rows, D, eps, dtype, false, stream);
}

kda_status_t kda_rms_norm_e4m3(const void *x, const void *residual, const float *weight, void *y, float *scale, void *h,
                               long long rows, int D, float eps, kda_dtype_t dtype, void *stream)
{
    return run_norm(x, residual, weight, y, scale, h, rows, D, eps, dtype, true, stream);
}

size_t kda_rms_norm_bwd_workspace_size(long long rows, int D)
{
    if (rows < 0 || rows > 0x7fffffffLL || D <= 0 || D % 8 != 0 || D > kNormMaxWidth) return 0;
    const int a = bwd_blocks(rows, D / 8), b = bwd_blocks(rows, D / 4);      // bf16, fp32
    return (size_t)(a > b ? a : b) * D * sizeof(float);
}

kda_status_t kda_rms_norm_bwd(const void *dy, const void *h, const float *weight, const void *dh, void *dx,
                              float *dweight, long long rows, int D, float eps, kda_dtype_t dtype, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (rows < 0 || D <= 0 || !(eps >= 0.f) || eps > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > kNormMaxWidth || rows > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (!dweight || !al(dweight, 16)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) return cudaMemsetAsync(dweight, 0, (size_t)D * 4, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    if (!dy || !h || !weight || !dx || !workspace) return KDA_ERR_INVALID_ARG;
    if (!al(dy, 16) || !al(h, 16) || !al(weight, 16) || !al(dh, 16) || !al(dx, 16) || !al(workspace, 16))
        return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda_rms_norm_bwd_workspace_size(rows, D)) return KDA_ERR_INVALID_ARG;
    NormBwdParams p;
    p.dy = dy; p.h = h; p.dh = dh; p.w = weight; p.dx = dx; p.partial = (float *)workspace; p.eps = eps;
    p.inv_d = 1.f / (float)D; p.rows = rows; p.D = D;
    const int blocks = bwd_blocks(rows, dtype == KDA_BF16 ? D / 8 : D / 4);
    using bf = __nv_bfloat16;
    const cudaError_t e = dtype == KDA_BF16 ? (dh ? launch_norm_bwd<bf, true>(p, blocks, st) : launch_norm_bwd<bf, false>(p, blocks, st))
                                            : (dh ? launch_norm_bwd<float, true>(p, blocks, st) : launch_norm_bwd<float, false>(p, blocks, st));
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    // scheduled while the first kernel's last rows are worked on; it waits for all of them
    return launch_after(rms_norm_dw_kernel, (D + 31) / 32, 1024, 0, st, p.partial, dweight, blocks, D) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_latent_append(const void *c, const void *k_shared, const long long *slots, const float *weight,
                               void *cache, long long c_token_stride, long long shared_token_stride,
                               long long cache_rows, int T, int dc, int dr, float eps, kda_dtype_t dtype, void *stream)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (T < 0 || cache_rows < 0 || !(eps >= 0.f) || eps > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 || dc != kLatentDim || (dr != 0 && dr != kSharedDim)) return KDA_ERR_UNSUPPORTED;
    if (T == 0) return KDA_OK;
    if (!c || !slots || !cache || (dr && !k_shared)) return KDA_ERR_INVALID_ARG;
    if (!al(c, 16) || !al(slots, 8) || !al(cache, 16) || !al(weight, 16)) return KDA_ERR_INVALID_ARG;
    if (c_token_stride % 8 != 0 || c_token_stride < 0) return KDA_ERR_INVALID_ARG;
    if (dr && (!al(k_shared, 16) || shared_token_stride % 8 != 0 || shared_token_stride < 0)) return KDA_ERR_INVALID_ARG;
    const cudaError_t e = launch_after(latent_append_kernel, (T + 3) / 4, 128, 0, (cudaStream_t)stream, (const __nv_bfloat16 *)c,
                                       (const __nv_bfloat16 *)k_shared, slots, weight, (__nv_bfloat16 *)cache, c_token_stride,
                                       shared_token_stride, cache_rows, T, dr, eps);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
