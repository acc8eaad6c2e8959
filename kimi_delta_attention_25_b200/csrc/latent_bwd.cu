// latent_bwd.cu -- the backward pass of the expanded latent attention (latent_fwd.cu), with P recomputed
// from the forward's lse:  P = exp(s - lse),  D_i = do_i . o_i,  dP = do v^T,  dS = P (dP - D),
//   dq = scale dS [k, r],  dk = scale dS^T q[:128],  dr = scale sum_h dS^T q[128:],  dv = P^T do.
//
// Two kinds of blocks, each for one row of tiles, none of them adding to memory that another block adds to:
//   dq:        rows of 128 queries, over key tiles:   S = Q [K, R]^T, dP = dO V^T,     dq += dS [K, R]
//   dk and dv: rows of 128 keys, over query tiles:    S^T = [K, R] Q^T, dP^T = V dO^T, dk, dr += dS^T Q, dv += P^T dO
// A fused dq would need atomic sums, or dS through memory (2.1 GB written and read for 8192 tokens x 16 heads, 330 us,
// where computing S and dP again takes 160).
// The tensor cores bound it: per 128 x 128 tile and head 804 + 536 + 792 cycles for dq and 804 + 3 x 536 + 280 for dk and
// dv, 4820 in all, where a single pass without the recomputation would take 3460. Measured: 2690 for dq and 3650 for dk
// and dv, where each tile's chain of scores, exponentials and P's product is the longer; 8192 tokens x 16 heads, causal,
// 0.96 to 0.99 ms alone, 1.10 to 1.12 under the power cap.
// dS and P pass through tensor memory in bf16 as A operands; sums, lse and D are fp32.
#include "latent.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int TL = 128;                       // rows and columns of a tile
constexpr int NT = 8 * 32 + 96, W_LOAD = 8, W_MMA = 9;   // warp 10: dq issues its accumulation there, dk and dv fetch statistics
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
// tokens): one warp per head and eight tokens, half a warp to a row, all its rows on their way at once (two tokens to a
// warp took twice the time).
// `out` has been rounded to bf16, which moves D by up to 2^-8 of |do| . |o|, and dS = P (dP - D) by P times that. Beside
// the rounding of dS itself that matters where one key has most of a row's probability (dS is then a difference of nearly
// equal values, and o as large as v). Rows that see at most kShortRow keys, where that is the rule, get D = sum_j P_ij dP_ij
// instead, from the same sums in fp32. A longer row that one key takes (P near 1) keeps D from `out`: recomputing D for all
// rows would take scores and dP once more, a quarter of the products there are.
constexpr int kShortRow = 16, kStatTokens = 8;
static_assert(8 * kStatTokens <= 64, "a block's tokens, a bit each");
__global__ void __launch_bounds__(256) latent_stat_kernel(LatentArgs a, const __nv_bfloat16 *__restrict__ dout, float *__restrict__ stat,
                                                          long long tokens)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0) check_call(a);
    __shared__ uint32_t short_of[8];           // bit = token of that warp that sees 2 to kShortRow keys
    __shared__ long long short_k0[8 * kStatTokens];
    __shared__ int short_keys[8 * kStatTokens];
    __shared__ float short_lse[8 * kStatTokens];
    const int H = a.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.x % H;
    const long long block0 = (long long)(blockIdx.x / H) * 8 * kStatTokens, t0 = block0 + warp * kStatTokens, tok = t0 + (lane & (kStatTokens - 1));
    uint4 o[kStatTokens / 2], od[kStatTokens / 2];
#pragma unroll
    for (int u = 0; u < kStatTokens / 2; ++u) {
        const long long t = t0 + 2 * u + (lane >> 4);
        o[u] = od[u] = make_uint4(0, 0, 0, 0);
        if (t < tokens) {
            o[u] = reinterpret_cast<const uint4 *>(a.out + (t * H + h) * kHeadDim)[lane & 15];
            od[u] = reinterpret_cast<const uint4 *>(dout + (t * H + h) * kHeadDim)[lane & 15];
        }
    }
    // from here a lane has a token: its lse, the keys that it sees, its sum
    const bool real = lane < kStatTokens && tok < tokens;
    const float l = real ? a.lse[tok * H + h] : 0.f;
    long long k0 = 0, seen = 0;
    if (real) {
        const int n = latent_sequence(a.cu_q, a.N, a.T, tok);
        LatentSpan s;
        if (n >= 0 && latent_span(a.cu_q, a.cu_k, n, a.T, a.Tk, &s)) {
            k0 = s.k0;
            seen = s.k1 - s.k0;
            if (a.causal) seen = min(seen, tok - s.q0 + (s.k1 - s.k0) - (s.q1 - s.q0) + 1);
        }
    }
    float mine = 0.f;
#pragma unroll
    for (int u = 0; u < kStatTokens / 2; ++u) {
        float x = dot8(o[u], od[u]);
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
        x = __shfl_sync(0xffffffffu, x, (lane & 1) * 16);
        if (lane >> 1 == u) mine = x;
    }
    const bool is_short = seen > 1 && seen <= kShortRow;
    const uint32_t shorts = __ballot_sync(0xffffffffu, is_short);
    if (real) {
        stat[(long long)h * tokens + tok] = l == -INFINITY ? INFINITY : l * 1.44269504088896341f;
        if (!is_short) stat[tokens * H + (long long)h * tokens + tok] = mine;
    }
    if (lane == 0) short_of[warp] = shorts;
    if (is_short) {
        const int i = warp * kStatTokens + lane;
        short_k0[i] = k0;
        short_keys[i] = (int)seen;
        short_lse[i] = l;
    }
    __syncthreads();
    // the block's short rows, dealt out to its warps (a sequence's first rows are all short)
    unsigned long long todo = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) todo |= (unsigned long long)short_of[w] << (w * kStatTokens);
    for (int turn = 0; todo; ++turn, todo &= todo - 1) {
        if ((turn & 7) != warp) continue;
        // eight lanes to a key, four keys at a time, every load of the row on its way at once
        const int i = __ffsll(todo) - 1, W = kHeadDim + a.R, part = lane & 7, cnt = short_keys[i];
        const long long t = block0 + i, first = short_k0[i];
        const float li = short_lse[i];
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
        if (lane == 0) stat[tokens * H + (long long)h * tokens + t] = sum;
    }
}

// What the blocks share: the tensor maps, the barriers' place, and the wait.
constexpr uint32_t OFF_BAR = 14 * UNIT + 2048, SMEM = OFF_BAR + 320;
static_assert(SMEM <= SMEM_MAX, "shared memory");
constexpr int kMaxBars = 36;
struct BwdMaps { CUtensorMap q, k, r, v, d; };

__device__ __forceinline__ volatile int *control(unsigned char *sm)          // [0] tensor memory, [1] abort
{
    return reinterpret_cast<volatile int *>(reinterpret_cast<uint64_t *>(sm + OFF_BAR) + kMaxBars);
}
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > 2000000000LL) { *abort_flag = 1; set_status(status, KDA_ERR_TIMEOUT); return false; }
    }
    return true;
}

// Results leave through shared memory: a lane has one row, and 16 bytes of 32 rows at a time is what a store writes worst
// (the end of a dq block took 7.6 thousand cycles that way, 3.6 so). C pieces of 16 bytes a row, rows of the stage one piece further apart.
template <int C>
__device__ __forceinline__ void stage_piece(unsigned char *stage, int lane, int piece, uint4 x)
{
    *reinterpret_cast<uint4 *>(stage + lane * (C * 16 + 16) + piece * 16) = x;
}
template <int C>
__device__ __forceinline__ void store_stage(const unsigned char *stage, int lane, int rows, void *dst, size_t pitch)
{
    __syncwarp();
#pragma unroll 4
    for (int i = lane; i < 32 * C; i += 32) {
        const int r = i / C, c = i % C;
        if (r < rows)
            *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(dst) + r * pitch + c * 16) =
                *reinterpret_cast<const uint4 *>(stage + r * (C * 16 + 16) + c * 16);
    }
    __syncwarp();
}
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// ------------------------------------------------------------------------------------------ dq
// The two warpgroups take halves of a result's row: C pieces of 16 bytes each.
template <int C>
__device__ __forceinline__ void dq_result(uint32_t acc, bool some, float scale, unsigned char *stage, int lane, int rows, __nv_bfloat16 *dst, size_t pitch)
{
#pragma unroll
    for (int c = 0; c < C / 4; ++c) {
        float o[32];
        if (some) tmem_ld32_sync(acc + c * 32, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = some ? o[e] * scale : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) stage_piece<C>(stage, lane, c * 4 + e, pack8(o + 8 * e));
    }
    store_stage<C>(stage, lane, rows, dst, pitch);
}
// Shared memory: Q (3 units) and dO (2) of the block's rows, a ring of 7 units for keys and one of 2 for values.
constexpr int N1 = 7, N2 = 2;
constexpr uint32_t G_A1 = 0, G_A2 = 3 * UNIT, G_B1 = 5 * UNIT, G_B2 = G_B1 + N1 * UNIT;
enum { G_RES, G_F1, G_E1 = G_F1 + N1, G_F2 = G_E1 + N1, G_E2 = G_F2 + N2, G_S = G_E2 + N2, G_SFREE, G_P, G_PFREE, G_DS,
       G_ACC, G_DRAIN, G_NBARS = G_DRAIN + 2 };
static_assert(G_NBARS <= kMaxBars, "barriers");
constexpr uint32_t TM_S = 0, TM_P = 128, TM_DS = 256, TM_ACC = 320;

// While dS(j) is formed from dP(j), S(j + 1) runs; while P(j + 1) is formed from it, the accumulating product of
// tile j and dP(j + 1) do. The units of B1 are freed one by one by the accumulation.
__device__ __forceinline__ void dq_block(const LatentArgs &a, const LatentBwdArgs &b, const LatentSpan &sp, long long r0, int h,
                                         const BwdMaps &maps, unsigned char *sm)
{
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long Lq = sp.q1 - sp.q0, Lk = sp.k1 - sp.k0, shift = Lk - Lq, row_first = sp.q0 + r0, rows = Lq - r0;
    // key tiles that some row of this one sees
    const long long keys = a.causal ? min(Lk, min(r0 + TL, Lq) + shift) : Lk;
    const int nt = keys > 0 ? (int)((keys + TL - 1) / TL) : 0;

    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile int *abort_flag = control(sm) + 1;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(control(sm));
    auto wait = [&](int x, uint32_t parity) { return wait_or_abort(&bars[x], parity, abort_flag, a.status); };
    const int u1 = 2 + (a.R ? 1 : 0);          // units of queries and of a tile of keys; dO and values have two

    if (warp == W_LOAD) {
        // ============================================================================ loader
        if (elect_one() && nt > 0) {
            mbar_arrive_expect_tx(&bars[G_RES], (u1 + 2) * UNIT);
            for (int u = 0; u < u1; ++u) tma_load_3d(sm + G_A1 + u * UNIT, &maps.q, &bars[G_RES], u * 64, (int)row_first, h);
            for (int u = 0; u < 2; ++u) tma_load_3d(sm + G_A2 + u * UNIT, &maps.d, &bars[G_RES], u * 64, (int)row_first, h);
            int s1 = 0, s2 = 0, used1 = 0, used2 = 0;
            uint32_t p1 = 0, p2 = 0;
            bool ok = true;
            for (int j = 0; j < nt && ok; ++j) {
                const int row = (int)(sp.k0 + (long long)j * TL);
                for (int u = 0; u < u1 && ok; ++u) {
                    if (used1 >= N1) ok = wait(G_E1 + s1, p1 ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars[G_F1 + s1], UNIT);
                    if (u < 2) tma_load_3d(sm + G_B1 + s1 * UNIT, &maps.k, &bars[G_F1 + s1], u * 64, row, h);
                    else tma_load_2d(sm + G_B1 + s1 * UNIT, &maps.r, &bars[G_F1 + s1], 0, row);
                    ++used1;
                    if (++s1 == N1) { s1 = 0; p1 ^= 1; }
                }
                for (int u = 0; u < 2 && ok; ++u) {
                    if (used2 >= N2) ok = wait(G_E2 + s2, p2 ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars[G_F2 + s2], UNIT);
                    tma_load_3d(sm + G_B2 + s2 * UNIT, &maps.v, &bars[G_F2 + s2], u * 64, row, h);
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
        float lse_r = 0.f, d_r = 0.f;
        if (real) { lse_r = st_lse[row_first + row]; d_r = st_d[row_first + row]; }
        // keys this row sees (a query that sees one key has P = 1 whatever its score: dS is 0, which dP - D would miss
        // by a rounding)
        long long hi = real ? Lk : 0;
        if (a.causal) hi = min(hi, r0 + row + shift + 1);
        if (hi == 1) hi = 0;
        const int hi_w = __reduce_min_sync(0xffffffffu, (int)max(hi, 0LL));
        for (int j = 0; j < nt; ++j) {
            const long long c0 = (long long)j * TL + g * 64;
            const bool edge = c0 + 64 > hi_w;
            const int hi_e = (int)max(0LL, min(64LL, hi - c0));
            wait(G_S, j & 1);
            __syncwarp();
            tc_fence_after();
            float p[64];
            tmem_ld64_sync(tmem + TM_S + lanes + g * 64, p);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[G_SFREE]);
#pragma unroll
            for (int e = 0; e < 64; ++e) p[e] = ex2(p[e] * sc - lse_r);
            // keys behind the sequence's end may be anything: zeros, before the accumulation reads them
            // (its rows are this tile's columns; each warpgroup clears its own)
            const int valid = (int)min((long long)TL, Lk - (long long)j * TL);
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
                for (int e = 0; e < 32; ++e) d[e] = p[half * 32 + e] * (d[e] - d_r);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (half * 32 + e >= hi_e) d[e] = 0.f;
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
        const int W = kHeadDim + a.R, half = W / 2;
        __nv_bfloat16 *dst = b.dq + ((size_t)(row_first + quad * 32) * a.H + h) * W + g * half;
        const size_t pitch = (size_t)a.H * W * sizeof(__nv_bfloat16);
        const int here = (int)min(32LL, max(0LL, rows - quad * 32));
        unsigned char *stage = sm + G_B1 + warp * 8192;       // the keys are done with
        if (a.R) dq_result<12>(tmem + TM_ACC + lanes + g * half, nt > 0, a.scale, stage, lane, here, dst, pitch);
        else dq_result<8>(tmem + TM_ACC + lanes + g * half, nt > 0, a.scale, stage, lane, here, dst, pitch);
    }
}

// ---------------------------------------------------------------------------------------- dk and dv
// Rows of 128 keys, over query tiles. Tensor memory holds S^T (128 columns), dP^T (128), dk and dv (128 each): the
// shared part's gradient, 64 columns more, does not fit as a sum, so its product of each tile goes to columns that
// the tile is done with and is added up in registers. P^T and dS^T are written in bf16 over the columns they came
// from, by each warpgroup over its own (words 0 .. 31 and 96 .. 127 of the region), which leaves columns 32 .. 95
// of dP's region for that product.
// One warp issues everything in this order: S(j + 1), dr(j), dk(j), dP(j + 1), dv(j + 1); the tensor cores run it in
// order, which is what keeps S(j + 1) behind dv(j) and dP(j + 1) behind dk(j). Meanwhile the warpgroups form dS(j)
// (beside S(j + 1)), P(j + 1) (beside dr(j) and dk(j)) and take dr(j) before dP(j + 1) overwrites it.
// Shared memory: K (3 units) and V (2) of the block's rows, two tiles of queries, one of dO, the statistics of the
// columns (two tiles of lse and D).
constexpr uint32_t K_A1 = 0, K_A2 = 3 * UNIT, K_B1 = 5 * UNIT, K_B2 = K_B1 + 6 * UNIT, K_STAT = 14 * UNIT;
static_assert(K_B2 + 2 * UNIT <= K_STAT && K_STAT + 2048 <= OFF_BAR, "shared memory");
enum { K_RES, K_F1, K_E1 = K_F1 + 2, K_F2 = K_E1 + 2, K_E2, K_S, K_P, K_PREADY, K_DS, K_DR, K_PFREE, K_ACC, K_STATF,
       K_STATE = K_STATF + 2, K_DRAIN = K_STATE + 2, K_NBARS };
static_assert((int)K_NBARS <= kMaxBars, "barriers");
constexpr uint32_t TK_S = 0, TK_P = 128, TK_DR = TK_P + 32, TK_DK = 256, TK_DV = 384;

__device__ __forceinline__ void dkv_block(const LatentArgs &a, const LatentBwdArgs &b, const LatentSpan &sp, long long r0, int h,
                                          const BwdMaps &maps, unsigned char *sm)
{
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long Lq = sp.q1 - sp.q0, Lk = sp.k1 - sp.k0, shift = Lk - Lq, row_first = sp.k0 + r0, rows = Lk - r0;
    // query tiles from the first that sees this tile's first key
    const long long q_lo = a.causal ? max(0LL, r0 - shift) : 0;
    const int t_lo = (int)(min(q_lo, Lq) / TL), nt = q_lo < Lq ? (int)((Lq + TL - 1) / TL) - t_lo : 0;

    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile int *abort_flag = control(sm) + 1;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(control(sm));
    auto wait = [&](int x, uint32_t parity) { return wait_or_abort(&bars[x], parity, abort_flag, a.status); };
    const bool has_r = a.R != 0;
    const int u1 = 2 + (has_r ? 1 : 0);

    if (warp == W_LOAD) {
        // ============================================================================ loader
        if (elect_one() && nt > 0) {
            mbar_arrive_expect_tx(&bars[K_RES], (u1 + 2) * UNIT);
            for (int u = 0; u < 2; ++u) {
                tma_load_3d(sm + K_A1 + u * UNIT, &maps.k, &bars[K_RES], u * 64, (int)row_first, h);
                tma_load_3d(sm + K_A2 + u * UNIT, &maps.v, &bars[K_RES], u * 64, (int)row_first, h);
            }
            if (has_r) tma_load_2d(sm + K_A1 + 2 * UNIT, &maps.r, &bars[K_RES], 0, (int)row_first);
            bool ok = true;
            int j = 0;
            for (; j < nt; ++j) {
                const int row = (int)(sp.q0 + (long long)(t_lo + j) * TL), x = j & 1;
                if (j >= 2 && !(ok = wait(K_E1 + x, ((j >> 1) - 1) & 1))) break;
                mbar_arrive_expect_tx(&bars[K_F1 + x], u1 * UNIT);
                for (int u = 0; u < u1; ++u) tma_load_3d(sm + K_B1 + (x * 3 + u) * UNIT, &maps.q, &bars[K_F1 + x], u * 64, row, h);
                if (j >= 1 && !(ok = wait(K_E2, (j - 1) & 1))) break;
                mbar_arrive_expect_tx(&bars[K_F2], 2 * UNIT);
                for (int u = 0; u < 2; ++u) tma_load_3d(sm + K_B2 + u * UNIT, &maps.d, &bars[K_F2], u * 64, row, h);
            }
            if (!ok) {                          // a wait ran out: what is in flight lands before the block ends
                mbar_wait(&bars[K_RES], 0, 100000000LL);
                for (int x = max(0, j - 1); x <= j && x < nt; ++x) mbar_wait(&bars[K_F1 + (x & 1)], (x >> 1) & 1, 100000000LL);
                if (j > 0) mbar_wait(&bars[K_F2], (j - 1) & 1, 100000000LL);
            }
        }
    } else if (warp == W_MMA) {
        // ======================================================================== MMA issuer
        const bool el = elect_one();
        constexpr uint32_t id_s = idesc_bf16(TL, TL, 0, 0), id_a = idesc_bf16(TL, 128, 0, 1), id_r = idesc_bf16(TL, 64, 0, 1);
        constexpr uint32_t hi = desc_hi(1024, SW_128B);
        const uint32_t a1_lo = desc_lo(sbase + K_A1, 16), a2_lo = desc_lo(sbase + K_A2, 16);
        const uint32_t b1_lo = desc_lo(sbase + K_B1, 16), b2_lo = desc_lo(sbase + K_B2, 16);     // as K-major operands
        const uint32_t q_lo_mn = desc_lo(sbase + K_B1, UNIT), d_lo_mn = desc_lo(sbase + K_B2, UNIT);
        const int ntu = __reduce_max_sync(0xffffffffu, nt);
        auto scores = [&](int j) {
            wait(K_F1 + (j & 1), (j >> 1) & 1);
            tc_fence_after();
            if (el) {
                const uint32_t y = b1_lo + (j & 1) * (3 * UNIT / 16);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    umma_ss(tmem + TK_S, desc64(a1_lo + (e >> 2) * (UNIT / 16) + (e & 3) * 2, hi),
                            desc64(y + (e >> 2) * (UNIT / 16) + (e & 3) * 2, hi), id_s, e > 0 ? 1 : 0);
                if (has_r) {
#pragma unroll
                    for (int e = 8; e < 12; ++e)
                        umma_ss(tmem + TK_S, desc64(a1_lo + (e >> 2) * (UNIT / 16) + (e & 3) * 2, hi),
                                desc64(y + (e >> 2) * (UNIT / 16) + (e & 3) * 2, hi), id_s, 1);
                }
                umma_commit(&bars[K_S]);
            }
        };
        auto dp = [&](int j) {
            wait(K_F2, j & 1);
            tc_fence_after();
            if (el) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    umma_ss(tmem + TK_P, desc64(a2_lo + (e >> 2) * (UNIT / 16) + (e & 3) * 2, hi),
                            desc64(b2_lo + (e >> 2) * (UNIT / 16) + (e & 3) * 2, hi), id_s, e > 0 ? 1 : 0);
                umma_commit(&bars[K_P]);
            }
        };
        if (ntu > 0) {
            wait(K_RES, 0);
            scores(0);
            dp(0);
        }
        for (int j = 0; j < ntu; ++j) {
            const uint32_t more = j > 0 ? 1 : 0;
            wait(K_PREADY, j & 1);
            tc_fence_after();
            if (el) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    umma_ts(tmem + TK_DV, tmem + TK_S + (e < 4 ? e * 8 : 64 + e * 8), desc64(d_lo_mn + e * 128, hi), id_a, e > 0 ? 1 : more);
                umma_commit(&bars[K_E2]);
            }
            if (j + 1 < ntu) scores(j + 1);
            wait(K_DS, j & 1);
            tc_fence_after();
            if (el) {
                const uint32_t y = q_lo_mn + (j & 1) * (3 * UNIT / 16);
                if (has_r) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        umma_ts(tmem + TK_DR, tmem + TK_P + (e < 4 ? e * 8 : 64 + e * 8), desc64(y + 2 * (UNIT / 16) + e * 128, hi), id_r, e > 0 ? 1 : 0);
                    umma_commit(&bars[K_DR]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    umma_ts(tmem + TK_DK, tmem + TK_P + (e < 4 ? e * 8 : 64 + e * 8), desc64(y + e * 128, hi), id_a, e > 0 ? 1 : more);
                umma_commit(&bars[K_E1 + (j & 1)]);
                umma_commit(&bars[K_ACC]);
            }
            if (j + 1 < ntu) {
                wait(K_PFREE, j & 1);
                dp(j + 1);
            }
            if (*abort_flag) break;
        }
        if (el) {
            umma_commit(&bars[K_DRAIN]);
            if (!mbar_wait(&bars[K_DRAIN], 0, 100000000LL)) set_status(a.status, KDA_ERR_TIMEOUT);
        }
    } else if (warp == W_MMA + 1) {
        // ====================================================== the columns' statistics, [buffer][group][lse, D][64]
        const long long tokens = (long long)a.B * a.T;
        const float *lse = b.stat + (size_t)h * tokens + sp.q0, *d = lse + (size_t)tokens * a.H;
        float *stat = reinterpret_cast<float *>(sm + K_STAT);
        for (int j = 0; j < nt; ++j) {
            float x[4], y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const long long c = (long long)(t_lo + j) * TL + e * 32 + lane;
                x[e] = c < Lq ? lse[c] : 0.f;
                y[e] = c < Lq ? d[c] : 0.f;
            }
            // The buffer's own barrier (one that completes every tile would not do: the warps may be done with tile j - 1
            // before this one looks for tile j - 2, and the parities are the same again)
            if (j >= 2) { wait(K_STATE + (j & 1), ((j >> 1) - 1) & 1); __syncwarp(); }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float *to = stat + (j & 1) * 256 + (e >> 1) * 128 + (e & 1) * 32 + lane;
                to[0] = x[e];
                to[64] = y[e];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[K_STATF + (j & 1)]);
        }
    } else if (warp < W_LOAD) {
        // ============================================================================ P and dS
        // Lane = key; the two warpgroups share the columns (queries).
        const int g = warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)quad << 21;
        const int row = quad * 32 + lane;
        const bool real = row < rows;
        const float sc = a.scale * 1.44269504088896341f;
        // queries that see this key: [lo, hi) of the sequence; [ds_lo, hi) with a gradient through the score (a query
        // that sees one key has none)
        const long long lo = a.causal ? r0 + row - shift : 0, hi = real ? Lq : 0;
        const long long ds_lo = Lk == 1 ? hi : a.causal && r0 + row == 0 ? max(lo, 1 - shift) : lo;
        const int lo_w = __reduce_max_sync(0xffffffffu, (int)max(ds_lo, 0LL)), hi_w = __reduce_min_sync(0xffffffffu, (int)hi);
        const float *stat = reinterpret_cast<const float *>(sm + K_STAT) + g * 128;
        float dr[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) dr[e] = 0.f;
        auto take_dr = [&](int j) {                          // the shared part's product of tile j
            wait(K_DR, j & 1);
            __syncwarp();
            tc_fence_after();
            float x[32];
            tmem_ld32_sync(tmem + TK_DR + lanes + g * 32, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) dr[e] += x[e];
        };
        for (int j = 0; j < nt; ++j) {
            const float *sj = stat + (j & 1) * 256;
            const long long c0 = (long long)(t_lo + j) * TL + g * 64;
            const bool edge = c0 < lo_w || c0 + 64 > hi_w;
            const int lo_e = (int)max(0LL, min(64LL, lo - c0)), hi_e = (int)max(0LL, min(64LL, hi - c0));
            const int ds_lo_e = (int)max(0LL, min(64LL, ds_lo - c0));
            wait(K_STATF + (j & 1), (j >> 1) & 1);
            wait(K_S, j & 1);
            __syncwarp();
            tc_fence_after();
            float p[64];
            tmem_ld64_sync(tmem + TK_S + lanes + g * 64, p);
            auto exps = [&](int from) {
#pragma unroll
                for (int e = from; e < from + 32; e += 4) {
                    const float4 l4 = *reinterpret_cast<const float4 *>(sj + e);
                    p[e] = ex2(p[e] * sc - l4.x);
                    p[e + 1] = ex2(p[e + 1] * sc - l4.y);
                    p[e + 2] = ex2(p[e + 2] * sc - l4.z);
                    p[e + 3] = ex2(p[e + 3] * sc - l4.w);
                }
            };
            exps(0);
            if (j > 0) {
                if (has_r) take_dr(j - 1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[K_PFREE]);
            }
            exps(32);
            if (edge) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e < lo_e || e >= hi_e) p[e] = 0.f;
            }
            // queries and gradients behind the sequence's end may be anything: zeros, before the products over them
            // (each warpgroup clears its own columns' rows; the scores' wait put both copies' earlier uses behind)
            const int valid = (int)min((long long)TL, Lq - (long long)(t_lo + j) * TL);
            if (valid < (g + 1) * 64) {
                const int from = max(valid, g * 64);
                wait(K_F2, j & 1);
                for (int u = 0; u < u1 + 2; ++u) {
                    unsigned char *un = sm + (u < u1 ? K_B1 + ((j & 1) * 3 + u) * UNIT : K_B2 + (u - u1) * UNIT);
                    for (int e = tid & 127; e < ((g + 1) * 64 - from) * 8; e += 128)
                        *reinterpret_cast<uint4 *>(un + from * 128 + e * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = pack_bf16x2(p[2 * e], p[2 * e + 1]);
            tmem_st32(tmem + TK_S + lanes + g * 96, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[K_PREADY]);
            wait(K_P, j & 1);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float d[32];
                tmem_ld32_sync(tmem + TK_P + lanes + g * 64 + half * 32, d);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 d4 = *reinterpret_cast<const float4 *>(sj + 64 + half * 32 + e);
                    const float *x = p + half * 32 + e;
                    d[e] = x[0] * (d[e] - d4.x);
                    d[e + 1] = x[1] * (d[e + 1] - d4.y);
                    d[e + 2] = x[2] * (d[e + 2] - d4.z);
                    d[e + 3] = x[3] * (d[e + 3] - d4.w);
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (half * 32 + e < ds_lo_e || half * 32 + e >= hi_e) d[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) w[half * 16 + e] = pack_bf16x2(d[2 * e], d[2 * e + 1]);
            }
            tmem_st32(tmem + TK_P + lanes + g * 96, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) { mbar_arrive(&bars[K_DS]); mbar_arrive(&bars[K_STATE + (j & 1)]); }
        }
        if (nt > 0) {
            if (has_r) take_dr(nt - 1);
            wait(K_ACC, (nt - 1) & 1);                       // and dv's products, which were issued before
            __syncwarp();
            tc_fence_after();
        }
        const size_t at = (size_t)(row_first + quad * 32) * a.H + h;
        const int here = (int)min(32LL, max(0LL, rows - quad * 32));
        unsigned char *stage = sm + K_B1 + warp * 16384;     // queries and dO are done with
        if (has_r) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float4 x = make_float4(dr[4 * e] * a.scale, dr[4 * e + 1] * a.scale, dr[4 * e + 2] * a.scale, dr[4 * e + 3] * a.scale);
                *reinterpret_cast<float4 *>(stage + lane * 144 + e * 16) = x;
            }
            store_stage<8>(stage, lane, here, b.dr_head + at * kSharedDim + g * 32, (size_t)a.H * kSharedDim * sizeof(float));
        }
        // one warpgroup writes dk, the other dv
        const float f = g ? 1.f : a.scale;
#pragma unroll
        for (int c = 0; c < kHeadDim; c += 32) {
            float o[32];
            if (nt > 0) tmem_ld32_sync(tmem + (g ? TK_DV : TK_DK) + lanes + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = nt > 0 ? o[e] * f : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) stage_piece<16>(stage, lane, c / 8 + e, pack8(o + 8 * e));
        }
        store_stage<16>(stage, lane, here, (g ? b.dv : b.dk) + at * kHeadDim, (size_t)a.H * kHeadDim * sizeof(__nv_bfloat16));
    }
}

// One launch for both: blocks of dk and dv, then of dq, so that the first kind's last blocks do not leave the GPU idle,
// each kind from a sequence's longest row of tiles to its shortest. (Ranking the tiles of all sequences, as the forward
// kernel does, cost these shorter blocks more than it gave: 105 us became 120, 6 sequences x 8 heads.)
__global__ void __launch_bounds__(NT, 1)
latent_bwd_kernel(LatentArgs a, LatentBwdArgs b, long long q_slots, long long k_slots, const __grid_constant__ BwdMaps maps)
{
    extern __shared__ __align__(1024) unsigned char sm[];
    const int h = blockIdx.x % a.H, warp = threadIdx.x >> 5;
    long long x = blockIdx.x / a.H;
    const bool keys = x < k_slots;
    if (!keys) x = q_slots - 1 - (x - k_slots);
    // tensor memory and barriers, beside the search for the block's tile
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile int *ctl = control(sm);
    if (warp == W_MMA) { tmem_alloc(const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(ctl)), 512); tmem_relinquish(); }
    if (warp == W_LOAD && elect_one()) {
        for (int i = 0; i < (keys ? (int)K_NBARS : (int)G_NBARS); ++i) {
            const bool by_warps = keys ? i == K_PREADY || i == K_DS || i == K_PFREE || i == K_STATE || i == K_STATE + 1 : i == G_SFREE || i == G_PFREE || i == G_DS;
            mbar_init(&bars[i], by_warps ? 8 : 1);
        }
        ctl[1] = 0;
        fence_mbar_init();
        if (a.T > 0 && a.Tk > 0) { tma_prefetch_desc(&maps.q); tma_prefetch_desc(&maps.k); tma_prefetch_desc(&maps.v); tma_prefetch_desc(&maps.d); }
    }
    // Inputs, offsets and statistics alike are read behind this wait only: that the statistics' kernel has waited for what
    // was before it makes those writes visible to its own threads, not to a kernel that overlaps it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.T == 0 && blockIdx.x == 0) check_call(a);               // (else the statistics' kernel does it)
    LatentSpan sp;
    long long r0;
    int n;
    bool some = latent_slot(keys ? a.cu_k : a.cu_q, a, keys ? a.Tk : a.T, keys, TL, x, &n, &sp, &r0);
    if (smem_u32(sm) & 1023u) {                // swizzled tiles need it (it holds)
        if (threadIdx.x == 0) set_status(a.status, KDA_ERR_CUDA);
        some = false;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl);
    if (some) {
        if (keys) dkv_block(a, b, sp, r0, h, maps, sm);
        else dq_block(a, b, sp, r0, h, maps, sm);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

// dr[key] = sum over heads of dr_head[key][h], in fp32 and in head order. 16 keys per block: 16 threads of a
// float4 each per key.
__global__ void __launch_bounds__(256) latent_dr_kernel(const float *__restrict__ dr_head, __nv_bfloat16 *__restrict__ dr, long long keys, int H)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const long long stat_blocks = (tokens + 8 * kStatTokens - 1) / (8 * kStatTokens) * a.H;
    const int W = kHeadDim + a.R;
    BwdMaps m = {};                                               // an empty side's tiles are never copied
    if (tokens > 0 && (!bf16_heads_map(&m.q, a.q, W, a.H, tokens, W, (long long)a.H * W, 64, TL) ||
                       !bf16_heads_map(&m.d, b.dout, kHeadDim, a.H, tokens, kHeadDim, (long long)a.H * kHeadDim, 64, TL)))
        return cudaErrorNotSupported;
    if (keys > 0 && (!bf16_heads_map(&m.k, a.k, kHeadDim, a.H, keys, a.k_head, a.k_tok, 64, TL) ||
                     !bf16_heads_map(&m.v, a.v, kHeadDim, a.H, keys, a.v_head, a.v_tok, 64, TL) ||
                     (a.R && !bf16_rows_map(&m.r, a.r, kSharedDim, keys, a.r_tok, 64, TL))))
        return cudaErrorNotSupported;
    const cudaError_t e = cudaFuncSetAttribute(latent_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    if (e != cudaSuccess) return e;
    cudaError_t err = cudaSuccess;
    if (tokens > 0)
        err = launch_after(latent_stat_kernel, (unsigned)stat_blocks, 256, 0, stream, a, b.dout, b.stat, tokens);
    // its blocks set themselves up while the statistics are being finished
    if (err == cudaSuccess)
        err = launch_after(latent_bwd_kernel, (unsigned)((q_slots + k_slots) * a.H), NT, SMEM, stream, a, b, q_slots, k_slots, m);
    if (err == cudaSuccess && a.R && keys > 0)
        err = launch_after(latent_dr_kernel, (unsigned)((keys + 15) / 16), 256, 0, stream, b.dr_head, b.dr, keys, a.H);
    return err;
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
    const long long tokens = (long long)B * T, keys = (long long)B * Tk;
    if ((tokens / TL + keys / TL + 2LL * N) * H > 0x7fffffffLL || (tokens / (8 * kStatTokens) + 1) * H > 0x7fffffffLL)
        return KDA_ERR_UNSUPPORTED;                               // blocks of a launch
    a.causal = causal != 0;
    LatentBwdArgs b;
    b.dout = (const __nv_bfloat16 *)dout;
    b.dq = (__nv_bfloat16 *)dq; b.dk = (__nv_bfloat16 *)dk_out; b.dv = (__nv_bfloat16 *)dv_out; b.dr = (__nv_bfloat16 *)dk_shared;
    b.stat = (float *)((unsigned char *)workspace + kStatusBytes);
    b.dr_head = (float *)((unsigned char *)b.stat + align256((size_t)B * T * H * 8));
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = N == 0 || B == 0 || (T == 0 && Tk == 0) ? launch_latent_check(a, st) : launch_latent_bwd(a, b, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
