// latent_fwd.cu -- the expanded form of the latent attention: softmax attention whose keys are a part
// per head (128 channels, expanded from the token's latent vector) and a part that all heads share (64
// channels, or none):  s_ij = scale (q_i[:128] . k_j + q_i[128:] . r_j),  o_i = sum_j softmax_j(s_ij) v_j.
// Packed sequences with their own numbers of queries and keys; with `causal` query i of Lq sees the keys
// up to i + Lk - Lq.
//
// The tensor cores bound it: 2 (192 + 128) flops per visible pair of tokens and head, where a score's
// exponential costs one of 16 a cycle: 1024 cycles per 128 x 128 tile beside 1340 of products. The kernel
// therefore works on two query tiles of 128 rows at once, one CTA per SM: while the tensor cores run one
// tile's products (S = Q K^T, then O += P V), the other tile's warpgroup computes its P.
//  - One row of a tile is one thread: the running maximum and sum need no exchange. S comes from tensor
//    memory into registers, P goes back over S's columns in bf16 and is the A operand of the second
//    product from there; O stays in tensor memory for the whole row of tiles (2 x (128 + 128) columns).
//  - The maximum moves only when the first half's sum or the second half's largest score passes it by 2^15
//    (P stays in range of bf16, l and O are fp32), so that O is rarely rescaled, and half of the row needs no
//    search for its maximum; the same threads do both.
//  - P is handed over in two halves, and the second product starts on the first while the second's
//    exponentials are being taken.
//  - The issuing and loading warps share their schedulers with the warps that take exponentials, which leave
//    them few slots: their loops are kept short (few barriers, the widest products),
//    and warp-uniform with one issuing thread, so that descriptors stay in uniform registers.
//  - Keys wait in a ring of four units (128 rows x 64 channels, the shared part a tile's third), freed one by one,
//    values in two whole tiles: with one of either the products waited for copies.
// Blocks run from the longest row of tiles to the shortest. 8192 tokens x 32 heads, causal: 532 to 541 us (1.27 PFLOP/s),
// 620 to 628 in a row of calls under the power cap; the tensor pipe is active for 57 % of the cycles. P's rounding to bf16
// is the operand type's; sums and statistics are fp32.
#include "latent.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int QT = 128, KT = 128;             // query rows of a tile (two per block), keys of a tile
constexpr int NT = 8 * 32 + 64, W_LOAD = 8, W_MMA = 9;
constexpr uint32_t UNIT = 16384;              // 128 rows x 64 channels, 128-byte swizzle
constexpr int NK = 4;                         // ring of key units
constexpr uint32_t OFF_Q = 0, OFF_K = 6 * UNIT, OFF_V = OFF_K + NK * UNIT, OFF_BAR = OFF_V + 4 * UNIT;   // two tiles of Q, the keys' ring, two tiles of V
constexpr uint32_t SMEM = OFF_BAR + 512 + 1024;
static_assert(SMEM <= 232448, "shared memory");
enum { B_Q, B_KF, B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + 2, B_S = B_VE + 2, B_PA = B_S + 2, B_PB = B_PA + 2, B_PV = B_PB + 2,
       B_DRAIN = B_PV + 2, N_BARS };
constexpr uint32_t TM_S = 0, TM_O = 256;      // S (and P over it) of the two tiles, O of the two tiles

__global__ void __launch_bounds__(NT, 1)
latent_fwd_kernel(LatentArgs a, long long slots, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % a.H;
    // tensor memory and barriers, beside the search for the block's tile
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile int *ctl = reinterpret_cast<volatile int *>(bars + N_BARS);      // [0] tensor memory, [1] abort
    if (warp == W_MMA) { tmem_alloc(const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(ctl)), 512); tmem_relinquish(); }
    if (tid == 0) {
        mbar_init(&bars[B_Q], 1);
        for (int i = 0; i < NK; ++i) { mbar_init(&bars[B_KF + i], 1); mbar_init(&bars[B_KE + i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[B_VF + i], 1);
            mbar_init(&bars[B_VE + i], 1);
            mbar_init(&bars[B_S + i], 1);
            mbar_init(&bars[B_PA + i], 4);
            mbar_init(&bars[B_PB + i], 4);
            mbar_init(&bars[B_PV + i], 1);
        }
        mbar_init(&bars[B_DRAIN], 1);
        ctl[1] = 0;
        fence_mbar_init();
        if (a.Tk > 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0) check_call(a);        // (other blocks set the status a second later at the earliest: a wait that ran out)
    LatentSpan span;
    long long r0;                              // the block's first row within its sequence
    bool some;
    if (a.N > 1 && slots <= kRankedSlots) {
        some = latent_ranked(a, 2 * QT, (int)slots, (int)(blockIdx.x / a.H), reinterpret_cast<int *>(sm), &span, &r0);
        fence_proxy_async_smem();
    } else {
        int n;
        some = latent_slot(a.cu_q, a, a.T, false, 2 * QT, slots - 1 - blockIdx.x / a.H, &n, &span, &r0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl);
    if (!some) {                               // uniform
        if (warp == W_MMA) tmem_dealloc(tmem, 512);
        return;
    }
    struct { long long q0, qn, k0, kn; } t = {span.q0 + r0, span.q1 - span.q0 - r0, span.k0, span.k1 - span.k0};
    // tiles of keys that some row of query tile i sees: row r of the sequence sees keys up to r + Lk - Lq
    const long long shift = t.kn - (span.q1 - span.q0);
    int nt[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long last = min(r0 + (i + 1) * QT, span.q1 - span.q0) - 1;      // the tile's last row
        long long keys = a.causal ? min(t.kn, last + shift + 1) : t.kn;
        if (i * QT >= t.qn || keys < 0) keys = 0;
        nt[i] = (int)((keys + KT - 1) / KT);
    }
    const int ntile = max(nt[0], nt[1]);

    volatile int *abort_flag = ctl + 1;
    auto wait = [&](int b, uint32_t parity) {
        if (mbar_try_wait(&bars[b], parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(&bars[b], parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > 2000000000LL) { *abort_flag = 1; set_status(a.status, KDA_ERR_TIMEOUT); return false; }
        }
        return true;
    };
    const int kunits = 2 + (a.R ? 1 : 0);      // units of a key tile; a value tile has two

    if (warp == W_LOAD) {
        // ============================================================================ loader
        if (elect_one() && ntile > 0) {
            mbar_arrive_expect_tx(&bars[B_Q], 2 * kunits * UNIT);
            for (int i = 0; i < 2; ++i)
                for (int u = 0; u < kunits; ++u)
                    tma_load_3d(sm + OFF_Q + (i * 3 + u) * UNIT, &tm_q, &bars[B_Q], u * 64, (int)(t.q0 + i * QT), h);
            bool ok = true;
            int j = 0, s = 0, used = 0;
            uint32_t ph = 0;
            for (; j < ntile; ++j) {
                const int row = (int)(t.k0 + (long long)j * KT), b = j & 1;
                for (int u = 0; u < kunits; ++u) {
                    if (used >= NK && !(ok = wait(B_KE + s, ph ^ 1))) break;
                    unsigned char *kd = sm + OFF_K + s * UNIT;
                    mbar_arrive_expect_tx(&bars[B_KF + s], UNIT);
                    if (u < 2) tma_load_3d(kd, &tm_k, &bars[B_KF + s], u * 64, row, h);
                    else tma_load_2d(kd, &tm_r, &bars[B_KF + s], 0, row);
                    ++used;
                    if (++s == NK) { s = 0; ph ^= 1; }
                }
                if (!ok || (j >= 2 && !(ok = wait(B_VE + b, ((j >> 1) - 1) & 1)))) break;
                unsigned char *vd = sm + OFF_V + b * 2 * UNIT;
                mbar_arrive_expect_tx(&bars[B_VF + b], 2 * UNIT);
                tma_load_3d(vd, &tm_v, &bars[B_VF + b], 0, row, h);
                tma_load_3d(vd + UNIT, &tm_v, &bars[B_VF + b], 64, row, h);
            }
            if (!ok) {                          // a wait ran out: what is in flight lands before the block ends
                mbar_wait(&bars[B_Q], 0, 100000000LL);
                for (int x = max(0, used - NK); x < used; ++x) mbar_wait(&bars[B_KF + x % NK], (x / NK) & 1, 100000000LL);
                for (int x = max(0, j - 2); x < j; ++x) mbar_wait(&bars[B_VF + (x & 1)], (x >> 1) & 1, 100000000LL);
            }
        }
    } else if (warp == W_MMA) {
        // ======================================================================== MMA issuer
        // The whole warp runs the loop and one thread issues: slots and addresses stay warp-uniform.
        const bool el = elect_one();
        constexpr uint32_t id_s = idesc_bf16(QT, KT, 0, 0), id_o = idesc_bf16(QT, 128, 0, 1);
        constexpr uint32_t hi = desc_hi(1024, SW_128B);
        const uint32_t q_lo = desc_lo(sbase + OFF_Q, 16), k_lo = desc_lo(sbase + OFF_K, 16), v_lo = desc_lo(sbase + OFF_V, UNIT);
        const int nt0 = __reduce_max_sync(0xffffffffu, nt[0]), nt1 = __reduce_max_sync(0xffffffffu, nt[1]);
        const int ntu = max(nt0, nt1);
        int ks = 0;                             // ring slot of the next key unit, its phase
        uint32_t kp = 0;
        // S of tile 0 (which waits for the units as they land), and of tile 1 (which frees them) if it has this one
        auto scores = [&](int i, bool mine) {
            int x = ks;
            uint32_t ph = kp;
            for (int u = 0; u < kunits; ++u) {
                if (i == 0) { wait(B_KF + x, ph); tc_fence_after(); }
                if (el) {
                    if (mine) {
                        const uint32_t q = q_lo + (i * 3 + u) * (UNIT / 16), k = k_lo + x * (UNIT / 16), d = tmem + TM_S + i * 128;
#pragma unroll
                        for (int e = 0; e < 4; ++e) umma_ss(d, desc64(q + e * 2, hi), desc64(k + e * 2, hi), id_s, (e > 0 || u > 0) ? 1 : 0);
                    }
                    if (i == 1) umma_commit(&bars[B_KE + x]);
                }
                if (++x == NK) { x = 0; ph ^= 1; }
            }
            if (el && mine) umma_commit(&bars[B_S + i]);
            if (i == 1) { ks = x; kp = ph; }
        };
        if (ntu > 0) {
            wait(B_Q, 0);
            scores(0, nt0 > 0);
            scores(1, nt1 > 0);
        }
        for (int j = 0; j < ntu; ++j) {
            const int b = j & 1;
            const bool more = j + 1 < ntu;
            wait(B_VF + b, (j >> 1) & 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int nti = i ? nt1 : nt0;
                if (j < nti) {
                    // O_i += P_i V, the first 64 keys and then the others
                    const uint32_t d = tmem + TM_O + i * 128, p = tmem + TM_S + i * 128, v = v_lo + b * (2 * UNIT / 16);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait((half ? B_PB : B_PA) + i, j & 1);
                        tc_fence_after();
                        if (el) {
#pragma unroll
                            for (int e = half * 4; e < half * 4 + 4; ++e)
                                umma_ts(d, p + e * 8, desc64(v + e * 128, hi), id_o, (e > 0 || j > 0) ? 1 : 0);
                        }
                    }
                    if (el) umma_commit(&bars[B_PV + i]);
                }
                if (i == 1 && el) umma_commit(&bars[B_VE + b]);
                if (more) scores(i, j + 1 < nti);
            }
            if (*abort_flag) break;
        }
        if (el) {
            umma_commit(&bars[B_DRAIN]);
            if (!mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) set_status(a.status, KDA_ERR_TIMEOUT);
        }
    } else {
        // ============================================================================ softmax
        const int i = warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)quad << 21;
        const uint32_t ts = tmem + TM_S + i * 128 + lanes, to = tmem + TM_O + i * 128 + lanes;
        const int row = i * QT + quad * 32 + lane;                  // of the block's 256
        const bool real = row < t.qn;
        const long long vis = a.causal ? min(t.kn, r0 + row + shift + 1) : t.kn;
        const int lim = real ? (int)max(0LL, vis) : 0;              // keys this row sees
        const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
        const int nti = nt[i];
        const float sc = a.scale * 1.44269504088896341f;
        float m = -1e30f, l = 0.f;
        for (int j = 0; j < nti; ++j) {
            wait(B_S + i, j & 1);
            __syncwarp();
            tc_fence_after();
            const int kb = j * KT;
            const bool edge = kb + KT > lim_warp;
            // P of 64 columns with the maximum so far, and its sum (taken in pairs). All exponentials go to the
            // special-function unit: a polynomial on the FMA units for a quarter of them cost more in issue slots,
            // which the issuing warps lack, than it saved (8K x 32 heads: 576 us where this takes 537).
            const uint64_t sc2 = f2(sc, sc);
            uint32_t w[32];
            auto load = [&](int c, float (&s)[64]) {
                tmem_ld64_sync(ts + c, s);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) s[e] = kb + c + e < lim ? s[e] : -INFINITY;
                }
            };
            auto exps = [&](const float (&s)[64]) {
                const uint64_t m2 = f2(-m, -m);
                uint64_t sum2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float x0, x1;
                    f2_split(f2_fma(f2(s[2 * e], s[2 * e + 1]), sc2, m2), x0, x1);
                    const float p0 = ex2(x0), p1 = ex2(x1);
                    sum2[e & 1] = f2_add(sum2[e & 1], f2(p0, p1));
                    w[e] = pack_bf16x2(p0, p1);
                }
                float s0, s1;
                f2_split(f2_add(sum2[0], sum2[1]), s0, s1);
                return s0 + s1;
            };
            auto publish = [&](int half) {                // over S's columns that are read already
                tmem_st32(ts + half * 32, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[(half ? B_PB : B_PA) + i]);
            };
            float s[64];
            load(0, s);
            float sum = exps(s);
            load(64, s);
            float t0 = max3(s[0], s[1], s[2]), t1 = max3(s[3], s[4], s[5]);
#pragma unroll
            for (int e = 6; e < 62; e += 4) { t0 = max3(t0, s[e], s[e + 1]); t1 = max3(t1, s[e + 2], s[e + 3]); }
            const float top_b = max3(t0, t1, fmaxf(s[62], s[63]));
            // A sum or a score that large (or not finite, or no maximum yet) means that the maximum has to move. Few
            // tiles come here: the row's maximum, O and l scaled to it, and the first half again.
            if (__any_sync(0xffffffffu, !(sum < 32768.f) || top_b * sc > m + 15.f)) {
                load(0, s);
                float top = top_b;
#pragma unroll
                for (int e = 0; e < 64; ++e) top = fmaxf(top, s[e]);
                const float up = fmaxf(m, top * sc), f = up == m ? 1.f : ex2(m - up);
                m = up;
                l *= f;
                if (j > 0) {
                    wait(B_PV + i, (j - 1) & 1);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {
                        float o[16];
                        tmem_ld16_sync(to + c, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st16(to + c, o);
                    }
                    tmem_st_wait();
                }
                sum = exps(s);
                load(64, s);
            }
            // values behind the sequence's last key may be anything: zeros, before the second product reads them
            if (kb + KT > t.kn) {
                const int valid = (int)(t.kn - kb);
                wait(B_VF + (j & 1), (j >> 1) & 1);
                for (int u = 0; u < 2; ++u)
                    for (int e = quad * 32 + lane; e < (KT - valid) * 8; e += 128)
                        *reinterpret_cast<uint4 *>(sm + OFF_V + ((j & 1) * 2 + u) * UNIT + valid * 128 + e * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            publish(0);
            sum += exps(s);
            publish(1);
            l += sum;
        }
        if (nti > 0) {
            wait(B_PV + i, (nti - 1) & 1);
            __syncwarp();
            tc_fence_after();
        }
        const size_t orow = (size_t)(t.q0 + row) * a.H + h;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
            float o[32];
            if (nti > 0) tmem_ld32_sync(to + c, o);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = nti > 0 ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
            if (real) {
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * kHeadDim + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
        }
        if (real) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

__global__ void __launch_bounds__(256) latent_check_kernel(LatentArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    check_call(a);
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
    if (cu_q && N == 0 && (T > 0 || Tk > 0)) return KDA_ERR_INVALID_ARG;       // tokens of no sequence
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

cudaError_t launch_latent_check(const LatentArgs &a, cudaStream_t stream)
{
    return launch_after(latent_check_kernel, 1, 256, 0, stream, a);
}

cudaError_t launch_latent_fwd(const LatentArgs &a, cudaStream_t stream)
{
    const long long tokens = (long long)a.B * a.T, keys = (long long)a.B * a.Tk, slots = tokens / (2 * QT) + a.N;
    const int W = kHeadDim + a.R;
    CUtensorMap tq = {}, tk = {}, tv = {}, tr = {};
    if (!bf16_heads_map(&tq, a.q, W, a.H, tokens, W, (long long)a.H * W, 64, QT)) return cudaErrorNotSupported;
    // without a key no copy is made
    if (keys > 0 && (!bf16_heads_map(&tk, a.k, kHeadDim, a.H, keys, a.k_head, a.k_tok, 64, KT) ||
                     !bf16_heads_map(&tv, a.v, kHeadDim, a.H, keys, a.v_head, a.v_tok, 64, KT) ||
                     (a.R && !bf16_rows_map(&tr, a.r, kSharedDim, keys, a.r_tok, 64, KT))))
        return cudaErrorNotSupported;
    const cudaError_t e = cudaFuncSetAttribute(latent_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(latent_fwd_kernel, (unsigned)(slots * a.H), NT, SMEM, stream, a, slots, tq, tk, tv, tr);
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
    if (((long long)B * T / (2 * QT) + N) * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;      // blocks of a launch
    const cudaError_t e = (long long)B * T == 0 || N == 0 ? launch_latent_check(a, st) : launch_latent_fwd(a, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
