// latent_bwd.cu -- the backward pass of the expanded latent attention (latent_fwd.cu), with P recomputed
// from the forward's lse:  P = exp(s - lse),  D_i = do_i . o_i,  dP = do v^T,  dS = P (dP - D),
//   dq = scale dS [k, r],  dk = scale dS^T q[:128],  dr = scale sum_h dS^T q[128:],  dv = P^T do.
//
// Three kinds of blocks, each for one row of tiles, none of them adding to memory that another block adds to:
//   dq: rows of 128 queries, over key tiles:    S = Q [K, R]^T, dP = dO V^T,     dq += dS [K, R]
//   dk: rows of 128 keys, over query tiles:     S^T = [K, R] Q^T, dP^T = V dO^T, dk += dS^T Q
//   dv: rows of 2 x 128 keys, over query tiles: S^T, dv += P^T dO
// (the first two are one template: resident operands A1, A2 and streamed ones B1, B2 swap roles). One block
// for dk and dv would need S^T, dP^T, dk (192 columns) and dv in tensor memory: 576 of 512 columns; with query
// tiles of 64, which fit, the products over 64 columns read their 128-row operand from shared memory twice as
// often and cost as much as computing S^T again. A fused dq would need atomic sums or 2 bytes of dS per pair in
// memory, read and written: about twice the time of recomputing S and dP.
// The tensor cores bound it: per 128 x 128 tile and head 804 + 536 + 792 cycles for dq and dk each and
// 804 + 536 for dv, 5600 in all, where a single pass without the recomputation would take 3460.
// dS (and P) pass through tensor memory in bf16 as A operands; sums, lse and D are fp32.
#include "latent.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int TL = 128;                       // rows and columns of a tile
constexpr int NT = 8 * 32 + 96, W_LOAD = 8, W_MMA = 9;   // two issuing warps (one takes longer than the tensor cores)
constexpr uint32_t UNIT = 16384;              // 128 rows x 64 channels, 128-byte swizzle
constexpr uint32_t SMEM_MAX = 232448;

// Eight bf16 products added up.
__device__ __forceinline__ float dot8(const uint4 &x, const uint4 &y)
{
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        s += __uint_as_float(a[e] << 16) * __uint_as_float(b[e] << 16);
        s += __uint_as_float(a[e] & 0xFFFF0000u) * __uint_as_float(b[e] & 0xFFFF0000u);
    }
    return s;
}

// lse in the log2 domain and D_i = do_i . o_i as [H][tokens] (the dk and dv blocks read them along the
// tokens): one warp per head and two tokens, half a warp to a row.
// `out` has been rounded to bf16, which moves D by up to 2^-8 of |do| . |o|. Beside the rounding of dS itself that
// matters where a row sees few keys (dS is then a difference of nearly equal values, and o as large as v): rows
// that see at most kShortRow keys get D = sum_j P_ij dP_ij instead, from the same sums in fp32.
constexpr int kShortRow = 16;
__global__ void __launch_bounds__(256) latent_stat_kernel(LatentArgs a, const __nv_bfloat16 *__restrict__ dout, float *__restrict__ stat,
                                                          long long tokens)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0) check_call(a);
    const int H = a.H, lane = threadIdx.x & 31, h = blockIdx.y;
    const long long t0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 2, tok = t0 + (lane >> 4);
    if (t0 >= tokens) return;
    const bool real = tok < tokens;
    uint4 o = make_uint4(0, 0, 0, 0), od = o;
    float l = 0.f;
    if (real) {
        o = reinterpret_cast<const uint4 *>(a.out + (tok * H + h) * kHeadDim)[lane & 15];
        od = reinterpret_cast<const uint4 *>(dout + (tok * H + h) * kHeadDim)[lane & 15];
        l = a.lse[tok * H + h];
    }
    long long k0 = 0, seen = 0;                // the keys that this half warp's token sees
    if (real) {
        const int n = latent_sequence(a.cu_q, a.N, a.T, tok);
        LatentSpan s;
        if (n >= 0 && latent_span(a.cu_q, a.cu_k, n, a.T, a.Tk, &s)) {
            k0 = s.k0;
            seen = s.k1 - s.k0;
            if (a.causal) seen = min(seen, tok - s.q0 + (s.k1 - s.k0) - (s.q1 - s.q0) + 1);
        }
    }
    float mine = dot8(o, od);
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, m);
    for (uint32_t todo = __ballot_sync(0xffffffffu, (lane & 15) == 0 && seen > 1 && seen <= kShortRow); todo; todo &= todo - 1) {
        // eight lanes to a key, four keys at a time, every load of the row on its way at once
        const int i = __ffs(todo) - 1, W = kHeadDim + a.R, part = lane & 7;
        const long long t = t0 + (i >> 4), first = __shfl_sync(0xffffffffu, k0, i);
        const int cnt = (int)__shfl_sync(0xffffffffu, seen, i);
        const float li = __shfl_sync(0xffffffffu, l, i);
        const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (t * H + h) * W), *d = reinterpret_cast<const uint4 *>(dout + (t * H + h) * kHeadDim);
        const uint4 q0 = q[part], q1 = q[8 + part], q2 = a.R ? q[16 + part] : make_uint4(0, 0, 0, 0), d0 = d[part], d1 = d[8 + part];
        float x[kShortRow / 4], dp[kShortRow / 4], sum = 0.f;
#pragma unroll
        for (int u = 0; u < kShortRow / 4; ++u) {
            const int j = 4 * u + (lane >> 3);
            x[u] = dp[u] = 0.f;
            if (j < cnt) {
                const uint4 *k = reinterpret_cast<const uint4 *>(a.k + (first + j) * a.k_tok + h * a.k_head);
                const uint4 *v = reinterpret_cast<const uint4 *>(a.v + (first + j) * a.v_tok + h * a.v_head);
                x[u] = dot8(q0, k[part]) + dot8(q1, k[8 + part]);
                if (a.R) x[u] += dot8(q2, reinterpret_cast<const uint4 *>(a.r + (first + j) * a.r_tok)[part]);
                dp[u] = dot8(d0, v[part]) + dot8(d1, v[8 + part]);
            }
        }
#pragma unroll
        for (int u = 0; u < kShortRow / 4; ++u) {
#pragma unroll
            for (int m = 4; m > 0; m >>= 1) {
                x[u] += __shfl_xor_sync(0xffffffffu, x[u], m);
                dp[u] += __shfl_xor_sync(0xffffffffu, dp[u], m);
            }
            if (4 * u + (lane >> 3) < cnt) sum += expf(x[u] * a.scale - li) * dp[u];
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (lane == i) mine = sum;
    }
    if (real && (lane & 15) == 0) {
        stat[(long long)h * tokens + tok] = l == -INFINITY ? INFINITY : l * 1.44269504088896341f;
        stat[tokens * H + (long long)h * tokens + tok] = mine;
    }
}

// ------------------------------------------------------------------------------------ dq and dk
// Shared memory: A1 (3 units), A2 (2), a ring of 7 units for B1 and one of 2 for B2, the statistics of the
// columns (dk: two tiles of 128 values of each kind).
constexpr int N1 = 7, N2 = 2;
constexpr uint32_t G_A1 = 0, G_A2 = 3 * UNIT, G_B1 = 5 * UNIT, G_B2 = G_B1 + N1 * UNIT, G_STAT = G_B2 + N2 * UNIT,
                   G_BAR = G_STAT + 2048, G_END = G_BAR + 320;
static_assert(G_END <= SMEM_MAX, "shared memory");
enum { G_RES, G_F1, G_E1 = G_F1 + N1, G_F2 = G_E1 + N1, G_E2 = G_F2 + N2, G_S = G_E2 + N2, G_SFREE, G_P, G_PFREE, G_DS,
       G_ACC, G_DRAIN, G_NBARS = G_DRAIN + 2 };
static_assert(G_NBARS * 8 + 16 <= 320, "barriers");
constexpr uint32_t TM_S = 0, TM_P = 128, TM_DS = 256, TM_ACC = 320;

struct GradMaps { CUtensorMap a1, a1r, a2, b1, b1r, b2; };   // dq: q, -, dout, k, r, v; dk: k, r, v, q, -, dout

// While dS(j) is formed from dP(j), S(j + 1) runs; while P(j + 1) is formed from it, the accumulating product of
// tile j and dP(j + 1) do. The units of B1 are freed one by one by the accumulation.
template <bool DQ>
__device__ __forceinline__ void grad_block(const LatentArgs &a, const LatentBwdArgs &b, const LatentSpan &sp, long long r0, int h,
                                           const GradMaps &maps, unsigned char *sm)
{
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long Lq = sp.q1 - sp.q0, Lk = sp.k1 - sp.k0, shift = Lk - Lq;
    const long long row_first = (DQ ? sp.q0 : sp.k0) + r0, rows = (DQ ? Lq : Lk) - r0;     // rows: may exceed the tile
    const long long col_first = DQ ? sp.k0 : sp.q0, cols = DQ ? Lk : Lq;
    // tiles of the other side that some row of this one meets
    int t_lo = 0, t_hi;
    if (DQ) {
        long long keys = a.causal ? min(Lk, min(r0 + TL, Lq) + shift) : Lk;
        t_hi = keys > 0 ? (int)((keys + TL - 1) / TL) : 0;
    } else {
        const long long q = a.causal ? max(0LL, r0 - shift) : 0;           // first query that sees the first key here
        t_lo = (int)(min(q, Lq) / TL);
        t_hi = q < Lq ? (int)((Lq + TL - 1) / TL) : t_lo;
    }
    const int nt = t_hi - t_lo;

    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G_BAR);
    volatile int *ctl = reinterpret_cast<volatile int *>(bars + G_NBARS);
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl);
    volatile int *abort_flag = ctl + 1;
    auto wait = [&](int x, uint32_t parity) {
        if (mbar_try_wait(&bars[x], parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(&bars[x], parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > 2000000000LL) { *abort_flag = 1; set_status(a.status, KDA_ERR_TIMEOUT); return false; }
        }
        return true;
    };
    const int u1 = 2 + (a.R ? 1 : 0);          // units of A1 and of a tile of B1; A2 and B2 have two

    if (warp == W_LOAD) {
        // ============================================================================ loader
        if (elect_one() && nt > 0) {
            // units of keys with their shared part, or of whole query rows
            auto load1 = [&](bool key_side, const CUtensorMap *m, const CUtensorMap *mr, unsigned char *dst, uint64_t *bar, int u, int row) {
                if (key_side && u == 2) tma_load_2d(dst, mr, bar, 0, row);
                else tma_load_3d(dst, m, bar, u * 64, row, h);
            };
            mbar_arrive_expect_tx(&bars[G_RES], (u1 + 2) * UNIT);
            for (int u = 0; u < u1; ++u) load1(!DQ, &maps.a1, &maps.a1r, sm + G_A1 + u * UNIT, &bars[G_RES], u, (int)row_first);
            for (int u = 0; u < 2; ++u) tma_load_3d(sm + G_A2 + u * UNIT, &maps.a2, &bars[G_RES], u * 64, (int)row_first, h);
            int s1 = 0, s2 = 0, used1 = 0, used2 = 0;
            uint32_t p1 = 0, p2 = 0;
            bool ok = true;
            for (int j = 0; j < nt && ok; ++j) {
                const int row = (int)(col_first + (long long)(t_lo + j) * TL);
                for (int u = 0; u < u1 && ok; ++u) {
                    if (used1 >= N1) ok = wait(G_E1 + s1, p1 ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars[G_F1 + s1], UNIT);
                    load1(DQ, &maps.b1, &maps.b1r, sm + G_B1 + s1 * UNIT, &bars[G_F1 + s1], u, row);
                    ++used1;
                    if (++s1 == N1) { s1 = 0; p1 ^= 1; }
                }
                for (int u = 0; u < 2 && ok; ++u) {
                    if (used2 >= N2) ok = wait(G_E2 + s2, p2 ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars[G_F2 + s2], UNIT);
                    tma_load_3d(sm + G_B2 + s2 * UNIT, &maps.b2, &bars[G_F2 + s2], u * 64, row, h);
                    ++used2;
                    if (++s2 == N2) { s2 = 0; p2 ^= 1; }
                }
            }
            if (!ok) {                          // a wait ran out: what is in flight lands before the block ends
                mbar_wait(&bars[G_RES], 0, 100000000LL);
                for (int i = max(0, used1 - N1); i < used1; ++i) mbar_wait(&bars[G_F1 + i % N1], (i / N1) & 1, 100000000LL);
                for (int i = max(0, used2 - N2); i < used2; ++i) mbar_wait(&bars[G_F2 + i % N2], (i / N2) & 1, 100000000LL);
            }
        }
    } else if (warp >= W_MMA) {
        // ======================================================================== MMA issuers
        // The first warp issues S and dP, the second the accumulation; barriers order them where they depend on
        // one another.
        const bool el = elect_one();
        constexpr uint32_t id_s = idesc_bf16(TL, TL, 0, 0), id_a = idesc_bf16(TL, 64, 0, 1);
        constexpr uint32_t hi = desc_hi(1024, SW_128B);
        const uint32_t b1_lo = desc_lo(sbase + G_B1, 16), b2_lo = desc_lo(sbase + G_B2, 16);
        const int ntu = __reduce_max_sync(0xffffffffu, nt);
        if (warp == W_MMA) {
            const uint32_t a1_lo = desc_lo(sbase + G_A1, 16), a2_lo = desc_lo(sbase + G_A2, 16);
            int s1 = 0, s2 = 0;
            uint32_t p1 = 0, p2 = 0;
            if (ntu > 0) wait(G_RES, 0);
            for (int j = 0; j < ntu; ++j) {
                if (j > 0) wait(G_SFREE, (j - 1) & 1);
                for (int u = 0; u < u1; ++u) {
                    wait(G_F1 + s1, p1);
                    tc_fence_after();
                    if (el) {
                        const uint32_t x = a1_lo + u * (UNIT / 16), y = b1_lo + s1 * (UNIT / 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            umma_ss(tmem + TM_S, desc64(x + e * 2, hi), desc64(y + e * 2, hi), id_s, (e > 0 || u > 0) ? 1 : 0);
                    }
                    if (++s1 == N1) { s1 = 0; p1 ^= 1; }
                }
                if (el) umma_commit(&bars[G_S]);
                if (j > 0) wait(G_PFREE, (j - 1) & 1);
                for (int u = 0; u < 2; ++u) {
                    wait(G_F2 + s2, p2);
                    tc_fence_after();
                    if (el) {
                        const uint32_t x = a2_lo + u * (UNIT / 16), y = b2_lo + s2 * (UNIT / 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            umma_ss(tmem + TM_P, desc64(x + e * 2, hi), desc64(y + e * 2, hi), id_s, (e > 0 || u > 0) ? 1 : 0);
                        umma_commit(&bars[G_E2 + s2]);
                    }
                    if (++s2 == N2) { s2 = 0; p2 ^= 1; }
                }
                if (el) umma_commit(&bars[G_P]);
                if (*abort_flag) break;
            }
        } else {
            int c1 = 0;
            for (int j = 0; j < ntu; ++j) {
                wait(G_DS, j & 1);                  // B1 is there: the scores that dS came from read it
                tc_fence_after();
                for (int u = 0; u < u1; ++u) {
                    if (el) {
                        const uint32_t y = b1_lo + c1 * (UNIT / 16);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            umma_ts(tmem + TM_ACC + u * 64, tmem + TM_DS + e * 8, desc64(y + e * 128, hi), id_a, (e > 0 || j > 0) ? 1 : 0);
                        umma_commit(&bars[G_E1 + c1]);
                    }
                    if (++c1 == N1) c1 = 0;
                }
                if (el) umma_commit(&bars[G_ACC]);
                if (*abort_flag) break;
            }
        }
        if (el) {
            uint64_t *drain = &bars[G_DRAIN + warp - W_MMA];
            umma_commit(drain);
            if (!mbar_wait(drain, 0, 100000000LL)) set_status(a.status, KDA_ERR_TIMEOUT);
        }
    } else {
        // ============================================================================ P and dS
        // Lane = row; the two warpgroups share the columns.
        const int g = warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)quad << 21;
        const int row = quad * 32 + lane;
        const bool real = row < rows;
        const float sc = a.scale * 1.44269504088896341f;
        const long long tokens = (long long)a.B * a.T;
        const float *st_lse = b.stat + (size_t)h * tokens, *st_d = st_lse + (size_t)tokens * a.H;
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the statistics' kernel, whose end this block may overlap
        float lse_r = 0.f, d_r = 0.f;                        // dq: this row's
        if (DQ && real) { lse_r = st_lse[row_first + row]; d_r = st_d[row_first + row]; }
        // columns this row meets: [lo, hi) of the sequence
        // (a query that sees one key has P = 1 whatever its score: dS is 0, which dP - D would miss by a rounding)
        long long lo = 0, hi = real ? cols : 0;
        if (DQ) {
            if (a.causal) hi = min(hi, r0 + row + shift + 1);
            if (hi == 1) hi = 0;
        } else {
            if (a.causal) lo = r0 + row > 0 ? r0 + row - shift : 1 - shift;
            if (Lk == 1) hi = 0;
        }
        const int lo_w = __reduce_max_sync(0xffffffffu, (int)max(lo, 0LL)), hi_w = __reduce_min_sync(0xffffffffu, (int)max(hi, 0LL));
        float *stat = reinterpret_cast<float *>(sm + G_STAT);
        // dk: each warpgroup keeps its columns' statistics, [buffer][group][lse, D][64]
        float next = 0.f;
        auto fetch = [&](int j) {
            const int t = tid & 127;
            const long long c = (long long)(t_lo + j) * TL + g * 64 + (t & 63);
            next = c < cols ? (t < 64 ? st_lse : st_d)[col_first + c] : 0.f;
        };
        if (!DQ && nt > 0) fetch(0);
        for (int j = 0; j < nt; ++j) {
            float *sj = stat + ((j & 1) * 2 + g) * 128;
            if (!DQ) {
                sj[tid & 127] = next;
                if (j + 1 < nt) fetch(j + 1);
                named_bar_sync(1 + g, 128);
            }
            const long long c0 = (long long)(t_lo + j) * TL + g * 64;
            const bool edge = c0 < lo_w || c0 + 64 > hi_w;
            wait(G_S, j & 1);
            __syncwarp();
            tc_fence_after();
            float p[64];
            tmem_ld64_sync(tmem + TM_S + lanes + g * 64, p);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[G_SFREE]);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                float4 l4 = make_float4(lse_r, lse_r, lse_r, lse_r);
                if (!DQ) l4 = *reinterpret_cast<const float4 *>(sj + e);
                p[e] = ex2(p[e] * sc - l4.x);
                p[e + 1] = ex2(p[e + 1] * sc - l4.y);
                p[e + 2] = ex2(p[e + 2] * sc - l4.z);
                p[e + 3] = ex2(p[e + 3] * sc - l4.w);
            }
            // rows of B1 behind the sequence's end may be anything: zeros, before the accumulation reads them
            // (its rows are this tile's columns; each warpgroup clears its own)
            const int valid = (int)min((long long)TL, cols - (long long)(t_lo + j) * TL);
            if (valid < (g + 1) * 64) {
                const int from = max(valid, g * 64);
                for (int u = 0; u < u1; ++u) {
                    unsigned char *un = sm + G_B1 + (uint32_t)((j * u1 + u) % N1) * UNIT;
                    for (int e = tid & 127; e < ((g + 1) * 64 - from) * 8; e += 128)
                        *reinterpret_cast<uint4 *>(un + from * 128 + e * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            wait(G_P, j & 1);
            __syncwarp();
            tc_fence_after();
            uint32_t w[32];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float d[32];
                tmem_ld32_sync(tmem + TM_P + lanes + g * 64 + half * 32, d);
                if (half) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[G_PFREE]);
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    float4 d4 = make_float4(d_r, d_r, d_r, d_r);
                    if (!DQ) d4 = *reinterpret_cast<const float4 *>(sj + 64 + half * 32 + e);
                    float *x = p + half * 32 + e;
                    d[e] = x[0] * (d[e] - d4.x);
                    d[e + 1] = x[1] * (d[e + 1] - d4.y);
                    d[e + 2] = x[2] * (d[e + 2] - d4.z);
                    d[e + 3] = x[3] * (d[e + 3] - d4.w);
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const long long c = c0 + half * 32 + e;
                        if (c < lo || c >= hi) d[e] = 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) w[half * 16 + e] = pack_bf16x2(d[2 * e], d[2 * e + 1]);
            }
            if (j > 0) { wait(G_ACC, (j - 1) & 1); __syncwarp(); }       // dS was last read by the product of tile j - 1
            tmem_st32(tmem + TM_DS + lanes + g * 32, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[G_DS]);
        }
        if (nt > 0) {
            wait(G_ACC, (nt - 1) & 1);
            __syncwarp();
            tc_fence_after();
        }
        // results: chunks of 32 columns, the two warpgroups in turn
        const size_t at = (size_t)(row_first + row) * a.H + h;
#pragma unroll 1
        for (int c = g * 32; c < u1 * 64; c += 64) {
            float o[32];
            if (nt > 0) tmem_ld32_sync(tmem + TM_ACC + lanes + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = nt > 0 ? o[e] * a.scale : 0.f;
            if (!real) continue;
            if (!DQ && c >= kHeadDim) {
                float4 *dst = reinterpret_cast<float4 *>(b.dr_head + at * kSharedDim + c - kHeadDim);
#pragma unroll
                for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            } else {
                uint4 *dst = reinterpret_cast<uint4 *>(DQ ? b.dq + at * (kHeadDim + a.R) + c : b.dk + at * kHeadDim + c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dst[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                        pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
            }
        }
    }
}

// ------------------------------------------------------------------------------------------ dv
// The forward kernel's structure with the roles of queries and keys exchanged and lse known: two key tiles at
// once, P^T over S^T's columns as the A operand of dv += P^T dO.
constexpr int NVQ = 4;                        // ring of query units; dO has two tiles
constexpr uint32_t V_A = 0, V_Q = 6 * UNIT, V_D = V_Q + NVQ * UNIT, V_STAT = V_D + 4 * UNIT, V_BAR = G_BAR;
static_assert(V_STAT + 1024 <= V_BAR, "shared memory");
enum { V_RES, V_QF, V_QE = V_QF + NVQ, V_DF = V_QE + NVQ, V_DE = V_DF + 2, V_S = V_DE + 2, V_PA = V_S + 2, V_PB = V_PA + 2, V_PV = V_PB + 2,
       V_DRAIN = V_PV + 2, V_NBARS };
static_assert((int)V_NBARS <= (int)G_NBARS, "barriers");
constexpr uint32_t TV_S = 0, TV_O = 256;

__device__ __forceinline__ void dv_block(const LatentArgs &a, const LatentBwdArgs &b, const LatentSpan &sp, long long r0, int h,
                                         const GradMaps &maps, unsigned char *sm)
{
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long Lq = sp.q1 - sp.q0, Lk = sp.k1 - sp.k0, shift = Lk - Lq, rows = Lk - r0;
    const long long row_first = sp.k0 + r0;
    // query tiles that see some key of tile i: from the first that sees its first key to the last
    int first[2];
    const int t_hi = (int)((Lq + TL - 1) / TL);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long q = a.causal ? max(0LL, r0 + i * TL - shift) : 0;
        first[i] = (q < Lq && i * TL < rows) ? (int)(q / TL) : t_hi;
    }
    const int t_lo = min(first[0], first[1]);                  // tile 1 starts no earlier than tile 0, or has no rows
    const int nt = t_hi - t_lo;

    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + V_BAR);
    volatile int *ctl = reinterpret_cast<volatile int *>(bars + G_NBARS);
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl);
    volatile int *abort_flag = ctl + 1;
    auto wait = [&](int x, uint32_t parity) {
        if (mbar_try_wait(&bars[x], parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(&bars[x], parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > 2000000000LL) { *abort_flag = 1; set_status(a.status, KDA_ERR_TIMEOUT); return false; }
        }
        return true;
    };
    const int u1 = 2 + (a.R ? 1 : 0);

    if (warp == W_LOAD) {
        // ============================================================================ loader
        if (elect_one() && nt > 0) {
            mbar_arrive_expect_tx(&bars[V_RES], 2 * u1 * UNIT);
            for (int i = 0; i < 2; ++i)
                for (int u = 0; u < u1; ++u) {
                    unsigned char *dst = sm + V_A + (i * 3 + u) * UNIT;
                    if (u == 2) tma_load_2d(dst, &maps.a1r, &bars[V_RES], 0, (int)(row_first + i * TL));
                    else tma_load_3d(dst, &maps.a1, &bars[V_RES], u * 64, (int)(row_first + i * TL), h);
                }
            int s = 0, used = 0, j = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (; j < nt; ++j) {
                const int row = (int)(sp.q0 + (long long)(t_lo + j) * TL), b = j & 1;
                for (int u = 0; u < u1; ++u) {
                    if (used >= NVQ && !(ok = wait(V_QE + s, ph ^ 1))) break;
                    mbar_arrive_expect_tx(&bars[V_QF + s], UNIT);
                    tma_load_3d(sm + V_Q + s * UNIT, &maps.b1, &bars[V_QF + s], u * 64, row, h);
                    ++used;
                    if (++s == NVQ) { s = 0; ph ^= 1; }
                }
                if (!ok || (j >= 2 && !(ok = wait(V_DE + b, ((j >> 1) - 1) & 1)))) break;
                unsigned char *dst = sm + V_D + b * 2 * UNIT;
                mbar_arrive_expect_tx(&bars[V_DF + b], 2 * UNIT);
                tma_load_3d(dst, &maps.b2, &bars[V_DF + b], 0, row, h);
                tma_load_3d(dst + UNIT, &maps.b2, &bars[V_DF + b], 64, row, h);
            }
            if (!ok) {
                mbar_wait(&bars[V_RES], 0, 100000000LL);
                for (int x = max(0, used - NVQ); x < used; ++x) mbar_wait(&bars[V_QF + x % NVQ], (x / NVQ) & 1, 100000000LL);
                for (int x = max(0, j - 2); x < j; ++x) mbar_wait(&bars[V_DF + (x & 1)], (x >> 1) & 1, 100000000LL);
            }
        }
    } else if (warp == W_MMA) {
        // ======================================================================== MMA issuer, as in the forward kernel
        const bool el = elect_one();
        constexpr uint32_t id_s = idesc_bf16(TL, TL, 0, 0), id_o = idesc_bf16(TL, 128, 0, 1);
        constexpr uint32_t hi = desc_hi(1024, SW_128B);
        const uint32_t a_lo = desc_lo(sbase + V_A, 16), q_lo = desc_lo(sbase + V_Q, 16), d_lo = desc_lo(sbase + V_D, UNIT);
        const int ntu = __reduce_max_sync(0xffffffffu, nt);
        const int f0 = __reduce_max_sync(0xffffffffu, first[0] - t_lo), f1 = __reduce_max_sync(0xffffffffu, first[1] - t_lo);
        int qs = 0;
        uint32_t qp = 0;
        auto scores = [&](int i, bool mine) {
            int x = qs;
            uint32_t ph = qp;
            for (int u = 0; u < u1; ++u) {
                if (i == 0) { wait(V_QF + x, ph); tc_fence_after(); }
                if (el) {
                    if (mine) {
                        const uint32_t k = a_lo + (i * 3 + u) * (UNIT / 16), q = q_lo + x * (UNIT / 16), d = tmem + TV_S + i * 128;
#pragma unroll
                        for (int e = 0; e < 4; ++e) umma_ss(d, desc64(k + e * 2, hi), desc64(q + e * 2, hi), id_s, (e > 0 || u > 0) ? 1 : 0);
                    }
                    if (i == 1) umma_commit(&bars[V_QE + x]);
                }
                if (++x == NVQ) { x = 0; ph ^= 1; }
            }
            if (el && mine) umma_commit(&bars[V_S + i]);
            if (i == 1) { qs = x; qp = ph; }
        };
        if (ntu > 0) {
            wait(V_RES, 0);
            scores(0, f0 == 0);
            scores(1, f1 == 0);
        }
        for (int j = 0; j < ntu; ++j) {
            const int b = j & 1;
            const bool more = j + 1 < ntu;
            wait(V_DF + b, (j >> 1) & 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int f = i ? f1 : f0;
                if (j >= f) {
                    const uint32_t d = tmem + TV_O + i * 128, p = tmem + TV_S + i * 128, v = d_lo + b * (2 * UNIT / 16);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait((half ? V_PB : V_PA) + i, (j - f) & 1);
                        tc_fence_after();
                        if (el) {
#pragma unroll
                            for (int e = half * 4; e < half * 4 + 4; ++e)
                                umma_ts(d, p + e * 8, desc64(v + e * 128, hi), id_o, (e > 0 || j > f) ? 1 : 0);
                        }
                    }
                    if (el) umma_commit(&bars[V_PV + i]);
                }
                if (i == 1 && el) umma_commit(&bars[V_DE + b]);
                if (more) scores(i, j + 1 >= f);
            }
            if (*abort_flag) break;
        }
        if (el) {
            umma_commit(&bars[V_DRAIN]);
            if (!mbar_wait(&bars[V_DRAIN], 0, 100000000LL)) set_status(a.status, KDA_ERR_TIMEOUT);
        }
    } else if (warp < W_LOAD) {
        // ============================================================================ P
        const int i = warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)quad << 21;
        const uint32_t ts = tmem + TV_S + i * 128 + lanes, to = tmem + TV_O + i * 128 + lanes;
        const int row = i * TL + quad * 32 + lane;                  // of the block's 256 keys
        const bool real = row < rows;
        const float sc = a.scale * 1.44269504088896341f;
        const float *st_lse = b.stat + (size_t)h * ((long long)a.B * a.T);
        asm volatile("griddepcontrol.wait;" ::: "memory");          // the statistics' kernel
        const long long lo = a.causal ? r0 + row - shift : 0;       // first query that sees this key
        const int lo_w = __reduce_max_sync(0xffffffffu, (int)max(lo, 0LL));
        float *stat = reinterpret_cast<float *>(sm + V_STAT) + i * TL;
        const int f = first[i];
        float next = 0.f;
        auto fetch = [&](int tile) {
            const long long c = (long long)tile * TL + (tid & 127);
            next = c < Lq ? -st_lse[sp.q0 + c] : -INFINITY;
        };
        if (f < t_hi) fetch(f);
        for (int tile = f; tile < t_hi; ++tile) {
            const int j = tile - f;
            named_bar_sync(1 + i, 128);                             // the last tile's statistics are read
            stat[tid & 127] = next;
            if (tile + 1 < t_hi) fetch(tile + 1);
            named_bar_sync(1 + i, 128);
            const long long c0 = (long long)tile * TL;
            const bool edge = c0 < lo_w || c0 + TL > Lq;
            wait(V_S + i, j & 1);
            __syncwarp();
            tc_fence_after();
            // gradients of rows behind the sequence's last query may be anything: zeros, before the product reads them
            // (behind the wait for the scores: the ring slots' earlier uses are over by then, so the parity is this use's)
            if (c0 + TL > Lq) {
                const int valid = (int)(Lq - c0), x = tile - t_lo;
                wait(V_DF + (x & 1), (x >> 1) & 1);
                for (int u = 0; u < 2; ++u) {
                    unsigned char *un = sm + V_D + ((x & 1) * 2 + u) * UNIT;
                    for (int e = quad * 32 + lane; e < (TL - valid) * 8; e += 128)
                        *reinterpret_cast<uint4 *>(un + valid * 128 + e * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float s[64];
                tmem_ld64_sync(ts + half * 64, s);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const long long c = c0 + half * 64 + e;
                        if (c < lo || c >= Lq) s[e] = -INFINITY;
                    }
                }
                uint32_t w[32];
                const uint64_t sc2 = f2(sc, sc);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 l4 = *reinterpret_cast<const float4 *>(stat + half * 64 + 2 * e);       // minus lse
                    float x0, x1, x2, x3;
                    f2_split(f2_fma(f2(s[2 * e], s[2 * e + 1]), sc2, f2(l4.x, l4.y)), x0, x1);
                    f2_split(f2_fma(f2(s[2 * e + 2], s[2 * e + 3]), sc2, f2(l4.z, l4.w)), x2, x3);
                    w[e] = pack_bf16x2(ex2(x0), ex2(x1));
                    w[e + 1] = pack_bf16x2(ex2(x2), ex2(x3));
                }
                tmem_st32(ts + half * 32, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[(half ? V_PB : V_PA) + i]);
            }
        }
        const int cnt = t_hi - f;
        if (cnt > 0) {
            wait(V_PV + i, (cnt - 1) & 1);
            __syncwarp();
            tc_fence_after();
        }
        const size_t at = (size_t)(row_first + row) * a.H + h;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
            float o[32];
            if (cnt > 0) tmem_ld32_sync(to + c, o);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = cnt > 0 ? pack_bf16x2(o[2 * e], o[2 * e + 1]) : 0u;
            if (real) {
                uint4 *dst = reinterpret_cast<uint4 *>(b.dv + at * kHeadDim + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
        }
    }
}

// One launch for the three: blocks of dv, then of dk, then of dq, so that a kind's last blocks do not leave the GPU
// idle and the longest blocks (dv: two tiles of rows) are not the last, each kind from a sequence's longest row of tiles
// to its shortest. (Ranking the tiles of all sequences, as the forward kernel does, cost these shorter blocks more than
// it gave: 105 us became 120, 6 sequences x 8 heads.)
__global__ void __launch_bounds__(NT, 1)
latent_bwd_kernel(LatentArgs a, LatentBwdArgs b, long long q_slots, long long k_slots, long long v_slots,
                  const __grid_constant__ GradMaps mq, const __grid_constant__ GradMaps mk)
{
    extern __shared__ __align__(1024) unsigned char sm[];
    if (blockIdx.x == 0 && a.T == 0) check_call(a);              // (else the statistics' kernel does)
    const int h = blockIdx.x % a.H, warp = threadIdx.x >> 5;
    long long x = blockIdx.x / a.H;
    int kind = 2;                              // 0 dq, 1 dk, 2 dv
    if (x >= v_slots) { x -= v_slots; kind = 1; }
    if (kind == 1 && x >= k_slots) { x -= k_slots; kind = 0; }
    const bool keys = kind > 0;
    // tensor memory and barriers, beside the search for the block's tile
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G_BAR);
    volatile int *ctl = reinterpret_cast<volatile int *>(bars + G_NBARS);      // [0] tensor memory, [1] abort
    if (warp == W_MMA) { tmem_alloc(const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(ctl)), 512); tmem_relinquish(); }
    if (warp == W_LOAD && elect_one()) {
        for (int i = 0; i < (kind == 2 ? V_NBARS : G_NBARS); ++i) {
            const bool by_warps = kind == 2 ? i >= V_PA && i < V_PV : i == G_SFREE || i == G_PFREE || i == G_DS;
            mbar_init(&bars[i], by_warps ? (kind == 2 ? 4 : 8) : 1);
        }
        ctl[1] = 0;
        fence_mbar_init();
        const GradMaps &m = kind == 0 ? mq : mk;
        if (a.T > 0 && a.Tk > 0) { tma_prefetch_desc(&m.a1); tma_prefetch_desc(&m.a2); tma_prefetch_desc(&m.b1); tma_prefetch_desc(&m.b2); }
    }
    const int tile = kind == 2 ? 2 * TL : TL;
    const long long slots = kind == 0 ? q_slots : kind == 1 ? k_slots : v_slots;
    LatentSpan sp;
    long long r0;
    int n;
    bool some = latent_slot(keys ? a.cu_k : a.cu_q, a, keys ? a.Tk : a.T, keys, tile, keys ? x : slots - 1 - x, &n, &sp, &r0);
    if (smem_u32(sm) & 1023u) {                // swizzled tiles need it (it holds)
        if (threadIdx.x == 0) set_status(a.status, KDA_ERR_CUDA);
        some = false;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl);
    if (!some) {
        // no block ends before the statistics' kernel has: what follows this kernel must not overtake that one
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else if (kind == 0) {
        grad_block<true>(a, b, sp, r0, h, mq, sm);
    } else if (kind == 1) {
        grad_block<false>(a, b, sp, r0, h, mk, sm);
    } else {
        dv_block(a, b, sp, r0, h, mk, sm);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
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
    const long long tokens = (long long)a.B * a.T, keys = (long long)a.B * a.Tk;
    const long long q_slots = tokens > 0 ? tokens / TL + a.N : 0, k_slots = keys > 0 ? keys / TL + a.N : 0;
    const long long v_slots = keys > 0 ? keys / (2 * TL) + a.N : 0;
    if ((q_slots + k_slots + v_slots) * a.H > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int W = kHeadDim + a.R;
    CUtensorMap q = {}, k = {}, r = {}, v = {}, d = {};          // an empty side's tiles are never copied
    if (tokens > 0 && (!bf16_heads_map(&q, a.q, W, a.H, tokens, W, (long long)a.H * W, 64, TL) ||
                       !bf16_heads_map(&d, b.dout, kHeadDim, a.H, tokens, kHeadDim, (long long)a.H * kHeadDim, 64, TL)))
        return cudaErrorNotSupported;
    if (keys > 0 && (!bf16_heads_map(&k, a.k, kHeadDim, a.H, keys, a.k_head, a.k_tok, 64, TL) ||
                     !bf16_heads_map(&v, a.v, kHeadDim, a.H, keys, a.v_head, a.v_tok, 64, TL) ||
                     (a.R && !bf16_rows_map(&r, a.r, kSharedDim, keys, a.r_tok, 64, TL))))
        return cudaErrorNotSupported;
    constexpr uint32_t smem = G_END;
    const cudaError_t e = cudaFuncSetAttribute(latent_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const GradMaps mq = {q, q, d, k, r, v}, mk = {k, r, v, q, q, d};
    if (tokens > 0)
        latent_stat_kernel<<<dim3((unsigned)((tokens + 15) / 16), a.H), 256, 0, stream>>>(a, b.dout, b.stat, tokens);
    // its blocks set up and load their first tiles while the statistics are being finished
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((q_slots + k_slots + v_slots) * a.H));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = tokens > 0 ? 1 : 0;
    const cudaError_t e2 = cudaLaunchKernelEx(&cfg, latent_bwd_kernel, a, b, q_slots, k_slots, v_slots, mq, mk);
    if (e2 != cudaSuccess) return e2;
    if (a.R && keys > 0) latent_dr_kernel<<<(unsigned)((keys + 15) / 16), 256, 0, stream>>>(b.dr_head, b.dr, keys, a.H);
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
    return kStatusBytes + align256((size_t)B * T * H * 8) + align256((size_t)B * Tk * H * dr * 4);
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
    b.stat = (float *)((unsigned char *)workspace + kStatusBytes);
    b.dr_head = (float *)((unsigned char *)b.stat + align256((size_t)B * T * H * 8));
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 0 || B == 0 || (T == 0 && Tk == 0)) return cudaMemsetAsync(workspace, 0, kStatusBytes, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    return launch_latent_bwd(a, b, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
