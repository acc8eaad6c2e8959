// latent_decode.cu -- the absorbed form of the latent attention, for one or a few new tokens per sequence
// over a paged cache. Cache row j holds the token's latent vector c_j (512) and its shared key part r_j (64,
// or none); every head reads the same rows, as keys and (the latent) as values:
//   s_j = scale (q[:512] . c_j + q[512:] . r_j),   o = sum_j softmax_j(s) c_j   (512 values per head).
// Token t of a sequence's Tq new ones (the last of its seq_len cached tokens) sees the rows up to its own.
//
// What bounds it: the cache, 1152 bytes a row, read once; with 32 query rows that is 60 flops a byte, an
// eighth of what the tensor cores could do meanwhile. So the kernel is built around the copies:
//  - The queries of a sequence (Tq x H rows, in groups of at most 64) stay in shared memory, and the cache
//    streams past them in tiles of 64 rows. One tile serves both products from the same shared memory: as
//    K-major A operand of S^T = C Q^T and as MN-major A operand of O^T = C^T P^T. O^T (512 x rows, fp32) needs
//    4 x rows tensor-memory columns, where O itself would need all 512 for any number of rows.
//  - The products are limited by what they read from shared memory (A 128 rows x 16 = 4 KB an instruction at
//    128 bytes a cycle), which the copies' writes share: S^T with M = 64 reads 3 KB where S = Q C^T with
//    M = 128 (rows behind the queries unused) reads 6 KB and took 52 cycles an instruction (256 sequences x 32
//    heads, 1.5 GB: 392 us, then 342 with nothing else changed; 253 to 268 now, 5.7 to 6.0 TB/s).
//  - A thread of the softmax has one cache row and 16 of the query rows. It goes on with the running maxima
//    it has and only checks, in the same barrier that the tile needs anyway, whether a score passed one of
//    them by more than 2^8 (P stays below 2^8, l is fp32): maxima across threads, and the rescaling of O^T in
//    tensor memory, are for the few tiles where one did.
//  - The tiles of all sequences form one list, cut into equal shares, one per SM, whatever the
//    sequences' lengths. A sequence that a cut runs through leaves partial results (unnormalised O, maximum,
//    sum, fp32), which a second kernel joins in order of the shares: no atomics, the same bits each time.
//    The groups of one sequence (more than 64 rows) take the same share at the same time on neighbouring
//    SMs, so that one of them finds the other's tile in L2.
// P is rounded to bf16 as the operand of the second product; sums and statistics are fp32.
#include "latent.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int KT = 64;                       // cache rows per tile
constexpr int kLanes = 148;                  // shares of the list of tiles: one per SM of a B200
constexpr int HP = 16;                       // query rows of one softmax thread
constexpr uint32_t SLOT = 16384;             // 64 cache rows x 128 latent channels: two 64-channel halves
constexpr uint32_t SH_SLOT = 8192;           // 64 cache rows x the 64 shared channels

// Shared memory for groups of RG query rows (32 or 64): queries (9 chunks of 64 channels), P^T twice (64 cache
// rows of RG values), the shared key parts twice, and a ring of latent slots in what is left (a tile is four).
template <int RG> struct Lay {
    static constexpr int WG = RG / HP;                            // softmax warpgroups
    static constexpr int NSOFT = 128 * WG, W_LOAD = 4 * WG, W_MMA = W_LOAD + 1, NT = NSOFT + 64;
    static constexpr uint32_t Q = 0, QCHUNK = RG * 128;
    static constexpr uint32_t P = 9 * QCHUNK, PBUF = KT * RG * 2;
    static constexpr uint32_t SH = P + 2 * PBUF;
    static constexpr uint32_t RING = SH + 2 * SH_SLOT;
    static constexpr int NSLOT = RG == 64 ? 7 : 10;
    static constexpr uint32_t RED = RING + NSLOT * SLOT;          // float [4][RG]: each quarter's maxima, then its sums
    static constexpr uint32_t FAC = RED + 4 * RG * 4;             // float [RG]: factors of the columns of O^T
    static constexpr uint32_t MAXS = FAC + RG * 4;                // float [RG]: running maxima at a segment's end
    static constexpr uint32_t BAR = MAXS + RG * 4;
    static constexpr uint32_t TOTAL = BAR + 512 + 1024;           // with room to align the base
    static_assert(TOTAL + 1024 <= 232448, "shared memory");
    static_assert(QCHUNK % 1024 == 0 && P % 1024 == 0 && PBUF % 1024 == 0, "swizzle atoms");
};

struct DecodeArgs {
    const int32_t *table, *lens;
    __nv_bfloat16 *out;
    float *lse;
    int N, Tq, H, R, page, box, pages, max_pages;   // box: rows per copy (divides the page and the tile)
    int G, L;                                       // groups of query rows, shares
    float scale_log2;
    float *part, *part_ml;                          // [L * G][2][RG][512], [L * G][2][RG][2]
    int32_t *meta, *errs;                           // [L][2] {sequence cut at the share's end or -1, its last share}, [L * G]
    int32_t *status;
};

enum { B_QFULL, B_QEMPTY, B_SHFULL, B_SHEMPTY = B_SHFULL + 2, B_SFULL = B_SHEMPTY + 2, B_SFREE = B_SFULL + 2,
       B_PREADY = B_SFREE + 2, B_PVDONE = B_PREADY + 2, B_FULL = B_PVDONE + 2, B_EMPTY = B_FULL + 10, B_DRAIN = B_EMPTY + 10,
       N_BARS };
static_assert(N_BARS * 8 + 64 <= 512, "barriers");

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Barrier of `nthreads` threads that tells each whether any of them holds.
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t nthreads, bool mine)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
                 "barrier.cta.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"(id), "r"(nthreads), "r"((uint32_t)mine) : "memory");
    return r != 0;
}

// 16 values of each of lanes 0..15 (and of 16..31 among themselves), combined over the lanes: lane i (i + 16) gets
// the result of value i. Each exchange halves the values a lane still has.
template <typename Op>
__device__ __forceinline__ float spread16(float (&v)[16], int lane, Op op)
{
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
        const bool upper = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = upper ? v[i] : v[i + w], keep = upper ? v[i + w] : v[i];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, w));
        }
    }
    return v[0];
}

__device__ __forceinline__ int tiles_of(const DecodeArgs &a, int n, int *len_out, bool *bad)
{
    const int len = a.lens[n];
    if (len < 0 || (long long)len > (long long)a.max_pages * a.page) { *bad = true; *len_out = 0; return 0; }
    *len_out = len;
    return (len + KT - 1) / KT;
}

template <int RG>
__global__ void __launch_bounds__(Lay<RG>::NT, 1)
latent_decode_kernel(DecodeArgs a, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c)
{
    using Y = Lay<RG>;
    constexpr int NT = Y::NT, NSOFT = Y::NSOFT, W_LOAD = Y::W_LOAD, W_MMA = Y::W_MMA;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int share = blockIdx.x / a.G, g = blockIdx.x % a.G;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Y::BAR);
    volatile int *ctl = reinterpret_cast<volatile int *>(bars + N_BARS);   // [0] tmem, [1] abort, [2] error, [3] n0, [4] off0, [5] prefix
    __shared__ int s_warp[NT / 32];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == W_MMA) { tmem_alloc(const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(ctl)), 512); tmem_relinquish(); }
    if (tid == 0) {
        mbar_init(&bars[B_QFULL], 1);
        mbar_init(&bars[B_QEMPTY], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[B_SHFULL + i], 1);
            mbar_init(&bars[B_SHEMPTY + i], 1);
            mbar_init(&bars[B_SFULL + i], 1);
            mbar_init(&bars[B_SFREE + i], 4 * Y::WG);
            mbar_init(&bars[B_PREADY + i], 4 * Y::WG);
            mbar_init(&bars[B_PVDONE + i], 1);
        }
        for (int i = 0; i < Y::NSLOT; ++i) { mbar_init(&bars[B_FULL + i], 1); mbar_init(&bars[B_EMPTY + i], 1); }
        mbar_init(&bars[B_DRAIN], 1);
        ctl[1] = 0; ctl[2] = 0; ctl[3] = a.N; ctl[4] = 0; ctl[5] = 0;
        fence_mbar_init();
        if (a.pages > 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_c); }     // (else they were not made)
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The list of tiles: each thread counts a run of sequences, then finds whether this share begins in it.
    const int per = (a.N + NT - 1) / NT, n_lo = min(a.N, tid * per), n_hi = min(a.N, n_lo + per);
    bool bad = false;
    int mine = 0;                                              // (the host sees to it that the list fits 31 bits)
    for (int n = n_lo; n < n_hi; ++n) { int len; mine += tiles_of(a, n, &len, &bad); }
    int upto = mine;                                           // inclusive sums: within the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) upto += s_warp[w];
        total += s_warp[w];
    }
    // shares that get tiles: with fewer tiles than shares one each, so that no share inside a cut sequence is empty;
    // the first `longer` shares have base + 1 tiles, the others base
    const uint32_t used = min(a.L, total), base = used ? (uint32_t)total / used : 0, longer = used ? (uint32_t)total % used : 0;
    const int ntiles = share < (int)used ? (int)(base + (share < (int)longer ? 1 : 0)) : 0;
    const int begin = (int)(share * base + min((uint32_t)share, longer));
    {
        int at = upto - mine;
        if (ntiles > 0 && begin >= at && begin < upto)
            for (int n = n_lo; n < n_hi; ++n) {
                int len;
                const int t = tiles_of(a, n, &len, &bad);
                if (begin < at + t) { ctl[3] = n; ctl[4] = begin - at; ctl[5] = at; break; }
                at += t;
            }
    }
    if (bad) ctl[2] = KDA_ERR_INVALID_ARG;
    const int rows = min(RG, a.Tq * a.H - g * RG);             // this group's query rows
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl);
    const uint32_t TM_O = tmem + 128;
    const int n0 = ctl[3], off0 = ctl[4];
    const int chunks = 8 + (a.R ? 1 : 0);

    volatile int *abort_flag = ctl + 1;
    auto wait = [&](int b, uint32_t parity) {
        if (mbar_try_wait(&bars[b], parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(&bars[b], parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > 2000000000LL) { *abort_flag = 1; ctl[2] = KDA_ERR_TIMEOUT; return false; }
        }
        return true;
    };

    if (warp == W_LOAD) {
        // ============================================================================ loader
        // The warp's lanes share a tile's copies: one per 64-channel half and box of rows.
        const int nb = KT / a.box, b = lane % nb;
        int it = 0, seg = 0, n = n0, off = off0, slots_used = 0, slot_next = 0, slot_phase = 0, left = ntiles;
        bool ok = true;
        while (left > 0 && ok) {
            int len;
            bool x = false;
            const int tiles = tiles_of(a, n, &len, &x), cnt = min(tiles - off, left);
            if (cnt <= 0) { ++n; off = 0; continue; }
            auto load_q = [&]() {
                if (lane == 0) mbar_arrive_expect_tx(&bars[B_QFULL], chunks * Y::QCHUNK);
                __syncwarp();
                if (lane < chunks) tma_load_2d(sm + Y::Q + lane * Y::QCHUNK, &tm_q, &bars[B_QFULL], lane * 64, n * a.Tq * a.H + g * RG);
            };
            if (seg == 0) load_q();
            // row coordinate of this lane's box in tile t; behind the last row, or on a page that is not there, the
            // copy starts behind the cache and reads zeros
            // (the table's entry is read a tile ahead and looked at when its turn comes)
            int row = off * KT + b * a.box, pi = row / a.page, po = row % a.page;
            const int32_t *tab = a.table + (size_t)n * a.max_pages;
            int entry = row < len ? tab[pi] : 0;
            for (int t = off; t < off + cnt && ok; ++t, ++it) {
                int c1 = a.pages * a.page;
                if (row < len) {
                    if (entry >= 0 && entry < a.pages) c1 = entry * a.page + po;
                    else ctl[2] = KDA_ERR_INVALID_ARG;
                }
                row += KT; po += KT;
                while (po >= a.page) { po -= a.page; ++pi; }
                if (row < len) entry = tab[pi];
                if (a.R) {
                    const int s = it & 1;
                    if (it >= 2) ok = wait(B_SHEMPTY + s, ((it >> 1) - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars[B_SHFULL + s], SH_SLOT);
                    __syncwarp();
                    if (lane < nb) tma_load_2d(sm + Y::SH + s * SH_SLOT + b * a.box * 128, &tm_c, &bars[B_SHFULL + s], kLatentDim, c1);
                }
                for (int c = 0; c < 4; ++c) {
                    const int i = slots_used, s = slot_next;
                    if (i >= Y::NSLOT) ok = wait(B_EMPTY + s, slot_phase ^ 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars[B_FULL + s], SLOT);
                    __syncwarp();
                    const int half = lane / nb;
                    if (half < 2) tma_load_2d(sm + Y::RING + s * SLOT + half * 8192 + b * a.box * 128, &tm_c, &bars[B_FULL + s], c * 128 + half * 64, c1);
                    slots_used = i + 1;
                    if (++slot_next == Y::NSLOT) { slot_next = 0; slot_phase ^= 1; }
                    if (c == 1 && t == off && seg > 0) {
                        // the sequence's queries, once the last segment's scores are done (not in front of the cache
                        // rows, which need not wait; not behind them all, as the ring may be too short for that)
                        ok = __all_sync(0xffffffffu, wait(B_QEMPTY, (seg - 1) & 1));
                        if (!ok) break;
                        load_q();
                    }
                }
            }
            ++seg; left -= cnt; ++n; off = 0;
        }
        for (int i = share; i < a.N; i += a.L) {               // idle slots: nothing to attend to
            int len;
            bool x = false;
            if (tiles_of(a, i, &len, &x) == 0) {
                const size_t r0 = (size_t)i * a.Tq * a.H + g * RG;
                for (int e = lane; e < rows * (kLatentDim / 8); e += 32)
                    reinterpret_cast<uint4 *>(a.out + r0 * kLatentDim)[e] = make_uint4(0, 0, 0, 0);
                for (int e = lane; e < rows; e += 32) a.lse[r0 + e] = -INFINITY;
            }
        }
        // copies still in flight (only after a wait ran out) land before the block ends
        if (!ok && lane == 0) {
            if (seg >= 0 && left > 0) for (int i = 0; i < 100 && !mbar_wait(&bars[B_QFULL], seg & 1, 1000000LL); ++i) {}
            for (int i = max(0, slots_used - Y::NSLOT); i < slots_used; ++i)
                mbar_wait(&bars[B_FULL + i % Y::NSLOT], (i / Y::NSLOT) & 1, 100000000LL);
            if (a.R) for (int i = max(0, it - 1); i <= it; ++i) mbar_wait(&bars[B_SHFULL + (i & 1)], (i >> 1) & 1, 100000000LL);
        }
    } else if (warp == W_MMA) {
        // ======================================================================== MMA issuer
        // Scores of tile jt and the second product of the tile before, in a fixed order: half of the scores, the
        // second product (whose P is ready by then, and whose end frees ring slots), the other half. The whole
        // warp runs the loop and one thread issues, so that slots and addresses stay warp-uniform: operands of a
        // product come from uniform registers, and moving them there one by one took 63 cycles a product.
        const bool el = elect_one();
        constexpr uint32_t id_s = idesc_bf16(KT, RG, 0, 0), id_o = idesc_bf16(128, RG, 1, 1);
        constexpr uint32_t hi = desc_hi(1024, SW_128B), hi_p = RG == 64 ? hi : desc_hi(512, SW_64B);
        // K-major operands (cache rows as keys, queries), and MN-major ones: the cache rows as values, and P^T,
        // whose RG values a row are one swizzle atom wide
        const uint32_t q_lo = desc_lo(sbase + Y::Q, 16), p_lo = desc_lo(sbase + Y::P, 16), sh_lo = desc_lo(sbase + Y::SH, 16);
        const uint32_t k_lo = desc_lo(sbase + Y::RING, 16), v_lo = desc_lo(sbase + Y::RING, 8192);
        const int ntile = __reduce_max_sync(0xffffffffu, ntiles);
        const uint32_t has_r = a.R != 0;
        int n = n0, off = off0, seg = 0, seg_left = 0;
        int sslot = 0, pslot = 0;
        uint32_t sphase = 0, first_s = 0, first_p = 0;
        auto scores = [&](int c0, int c1, uint32_t d) {
            for (int c = c0; c < c1; ++c) {
                wait(B_FULL + sslot, sphase);
                tc_fence_after();
                if (el) {
                    const uint32_t qc = q_lo + c * (2 * Y::QCHUNK / 16), kc = k_lo + sslot * (SLOT / 16);
                    const uint32_t more = has_r | (c > 0 ? 1u : 0u);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ss(d, desc64(kc + (ks >> 2) * 512 + (ks & 3) * 2, hi),
                                desc64(qc + (ks >> 2) * (Y::QCHUNK / 16) + (ks & 3) * 2, hi), id_s, ks > 0 ? 1 : more);
                }
                if (++sslot == Y::NSLOT) { sslot = 0; sphase ^= 1; }
            }
        };
        for (int jt = 0; jt <= ntile; ++jt) {
            const uint32_t d = tmem + (uint32_t)(jt & 1) * 64;
            if (jt < ntile) {
                if (jt >= 2) wait(B_SFREE + (jt & 1), (uint32_t)((jt >> 1) - 1) & 1);
                first_s = 0;
                if (seg_left == 0) {
                    int len, tiles;
                    bool x = false;
                    while ((tiles = tiles_of(a, n, &len, &x) - off) <= 0) { ++n; off = 0; }
                    seg_left = __reduce_max_sync(0xffffffffu, min(tiles, ntile - jt));
                    wait(B_QFULL, seg & 1);
                    first_s = 1;
                }
                if (has_r) {
                    const int sh = jt & 1;
                    wait(B_SHFULL + sh, (uint32_t)(jt >> 1) & 1);
                    tc_fence_after();
                    if (el) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_ss(d, desc64(sh_lo + sh * (SH_SLOT / 16) + ks * 2, hi),
                                    desc64(q_lo + 8 * Y::QCHUNK / 16 + ks * 2, hi), id_s, ks > 0);
                        umma_commit(&bars[B_SHEMPTY + sh]);
                    }
                }
                scores(0, 2, d);
            }
            if (jt > 0) {
                const int pb = (jt - 1) & 1;
                wait(B_PREADY + pb, (uint32_t)((jt - 1) >> 1) & 1);
                tc_fence_after();
                const uint32_t more = first_p ^ 1u, pd = p_lo + pb * (Y::PBUF / 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (el) {
                        const uint32_t vc = v_lo + pslot * (SLOT / 16);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_ss(TM_O + c * RG, desc64(vc + ks * 128, hi), desc64(pd + ks * (RG * 2), hi_p), id_o, ks > 0 ? 1 : more);
                        umma_commit(&bars[B_EMPTY + pslot]);
                    }
                    if (++pslot == Y::NSLOT) pslot = 0;
                }
                if (el) umma_commit(&bars[B_PVDONE + pb]);
            }
            if (jt < ntile) {
                scores(2, 4, d);
                if (el) umma_commit(&bars[B_SFULL + (jt & 1)]);
                if (--seg_left == 0) { if (el) umma_commit(&bars[B_QEMPTY]); ++seg; ++n; off = 0; }
            }
            first_p = first_s;
            if (*abort_flag) break;
        }
        if (el) {
            umma_commit(&bars[B_DRAIN]);
            if (!mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) ctl[2] = KDA_ERR_TIMEOUT;
        }
    } else {
        // ============================================================================ softmax
        // Warp w has the cache rows 16 (w % 4) .. of the tile, one for each of its first 16 lanes (where a product
        // with M = 64 leaves them), and the query rows 16 (w / 4) ..; of O^T every (RG / 16)-th 128-channel chunk
        // from w / 4 on, all 128 lanes.
        constexpr float kNone = -1e30f, kOff = 1e30f;        // no score yet; a row that is none
        const int quad = warp & 3, grp = warp >> 2;
        const uint32_t lanes = (uint32_t)quad << 21;
        const int key = quad * 16 + lane;                    // lanes below 16
        float *red = reinterpret_cast<float *>(sm + Y::RED), *fac = reinterpret_cast<float *>(sm + Y::FAC);
        float *mseg = reinterpret_cast<float *>(sm + Y::MAXS);
        int j = 0;                                           // tile of this share
        int n = n0, off = off0, left = ntiles, pfx = ctl[5]; // pfx: tiles before sequence n
        int cut_n = -1, cut_last = 0;
        while (left > 0) {
            int len;
            bool x = false;
            const int tiles = tiles_of(a, n, &len, &x), cnt = min(tiles - off, left);
            if (cnt <= 0) { ++n; off = 0; continue; }
            // running maxima (log2 domain; lane i < 16 also has row i's in m_l), this thread's part of the sums
            float m[HP], lsum[HP], m_l = lane < HP && grp * HP + lane < rows ? kNone : kOff;
#pragma unroll
            for (int i = 0; i < HP; ++i) { m[i] = grp * HP + i < rows ? kNone : kOff; lsum[i] = 0.f; }
            for (int t = off; t < off + cnt; ++t, ++j) {
                const int buf = (int)(j & 1);
                wait(B_SFULL + buf, (uint32_t)(j >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                float s[HP];
                tmem_ld16_sync(tmem + lanes + buf * 64 + grp * HP, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_SFREE + buf]);
                const int k = t * KT + key;
                if (lane >= 16) {
#pragma unroll
                    for (int i = 0; i < HP; ++i) s[i] = -INFINITY;
                } else if (t * KT + KT > len - a.Tq + 1) {   // a tile whose last rows some query row does not see
                    int h = (g * RG + grp * HP) % a.H, lim = len - a.Tq + 1 + (g * RG + grp * HP) / a.H;
#pragma unroll
                    for (int i = 0; i < HP; ++i) {
                        if (k >= lim) s[i] = -INFINITY;
                        if (++h == a.H) { h = 0; ++lim; }
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < HP; ++i) top = fmaxf(top, s[i] * a.scale_log2 - m[i]);
                // rows of the tile behind the sequence's end may hold anything: zeros, as values
                const int valid = len - t * KT;
                if (valid < KT) {
                    for (int c = 0; c < 4; ++c) {
                        unsigned char *slot = sm + Y::RING + (uint32_t)((j * 4 + c) % Y::NSLOT) * SLOT;
                        for (int i = warp * 32 + lane; i < 2 * (KT - valid) * 8; i += NSOFT) {
                            const int hf = i / ((KT - valid) * 8), o = i % ((KT - valid) * 8);
                            *reinterpret_cast<uint4 *>(slot + hf * 8192 + valid * 128 + o * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (bar_or(1, NSOFT, top > 8.f)) {           // the same outcome in all warps
                    float v[HP];
#pragma unroll
                    for (int i = 0; i < HP; ++i) v[i] = s[i];
                    const float mine16 = spread16(v, lane, [](float x, float y) { return fmaxf(x, y); });
                    if (lane < HP) red[quad * RG + grp * HP + lane] = mine16;
                    named_bar_sync(1, NSOFT);
                    float f_l = 1.f;
                    if (lane < HP) {
                        const float *r = red + grp * HP + lane;
                        const float up = fmaxf(m_l, fmaxf(fmaxf(r[0], r[RG]), fmaxf(r[2 * RG], r[3 * RG])) * a.scale_log2);
                        if (up != m_l) f_l = ex2(m_l - up);
                        m_l = up;
                        if (quad == 0) fac[grp * HP + lane] = f_l;
                    }
#pragma unroll
                    for (int i = 0; i < HP; ++i) {
                        m[i] = __shfl_sync(0xffffffffu, m_l, i);
                        lsum[i] *= __shfl_sync(0xffffffffu, f_l, i);
                    }
                    named_bar_sync(1, NSOFT);
                    if (t > off) {
                        wait(B_PVDONE + (buf ^ 1), (uint32_t)((j - 1) >> 1) & 1);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c = grp; c < 4; c += Y::WG) {
#pragma unroll 1
                            for (int q = 0; q < RG / 16; ++q) {
                                const uint32_t ad = TM_O + lanes + c * RG + q * 16;
                                float o[16];
                                tmem_ld16_sync(ad, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= fac[q * 16 + i];
                                tmem_st16(ad, o);
                            }
                        }
                        tmem_st_wait();
                        tc_fence_before();
                    }
                }
                // P's buffer was last read by the second product of tile j - 2
                if (j >= 2) { wait(B_PVDONE + buf, (uint32_t)((j >> 1) - 1) & 1); __syncwarp(); }
                if (lane < 16) {
                    unsigned char *pr = sm + Y::P + buf * Y::PBUF;
#pragma unroll
                    for (int c = 0; c < HP / 8; ++c) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = 8 * c + 2 * i;
                            const float p0 = ex2(s[e] * a.scale_log2 - m[e]), p1 = ex2(s[e + 1] * a.scale_log2 - m[e + 1]);
                            lsum[e] += p0;
                            lsum[e + 1] += p1;
                            w[i] = pack_bf16x2(p0, p1);
                        }
                        const uint32_t at = RG == 64 ? sw128_offset(key, grp * HP + 8 * c) : sw64_offset(key, grp * HP + 8 * c);
                        *reinterpret_cast<uint4 *>(pr + at) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_PREADY + buf]);
            }
            // -------- the segment's results
            // (lanes above 15 have added zeros)
            const float mine16 = spread16(lsum, lane, [](float x, float y) { return x + y; });
            if (lane < HP) {
                red[quad * RG + grp * HP + lane] = mine16;
                if (quad == 0) mseg[grp * HP + lane] = m_l;
            }
            wait(B_PVDONE + ((j - 1) & 1), (uint32_t)((j - 1) >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            named_bar_sync(1, NSOFT);
            const bool whole = off == 0 && cnt == tiles;
            const size_t r0 = (size_t)n * a.Tq * a.H + g * RG;
            const size_t pslot = (size_t)blockIdx.x * 2 + (off == 0 ? 1 : 0);
            if (tid < RG) {
                const float l = (red[tid] + red[RG + tid]) + (red[2 * RG + tid] + red[3 * RG + tid]), mm = mseg[tid];
                fac[tid] = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                if (tid < rows) {
                    if (whole) a.lse[r0 + tid] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.69314718055994531f;
                    else *reinterpret_cast<float2 *>(a.part_ml + (pslot * RG + tid) * 2) = make_float2(l == 0.f ? -INFINITY : mm, l);
                }
            }
            named_bar_sync(1, NSOFT);
#pragma unroll 1
            for (int c = grp; c < 4; c += Y::WG) {
                const int dim = c * 128 + quad * 32 + lane;
#pragma unroll 1
                for (int q = 0; q * 16 < rows; ++q) {
                    float o[16];
                    tmem_ld16_sync(TM_O + lanes + c * RG + q * 16, o);
                    const int upto = rows - q * 16;
                    if (whole) {
                        __nv_bfloat16 *dst = a.out + (r0 + q * 16) * kLatentDim + dim;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < upto) dst[i * kLatentDim] = __float2bfloat16_rn(o[i] * fac[q * 16 + i]);
                    } else {
                        float *dst = a.part + (pslot * RG + q * 16) * kLatentDim + dim;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < upto) dst[i * kLatentDim] = o[i];
                    }
                }
            }
            if (!whole && off == 0) {                        // cut at this share's end: who joins it
                cut_n = n;
                const uint32_t last = (uint32_t)(pfx + tiles - 1), head = longer * (base + 1);
                cut_last = (int)(last < head ? last / (base + 1) : longer + (last - head) / base);
            }
            tc_fence_before();
            named_bar_sync(1, NSOFT);                        // the sums and O are read before the next segment
            left -= cnt; pfx += tiles; ++n; off = 0;
        }
        if (tid == 0 && g == 0) { a.meta[2 * share] = cut_n; a.meta[2 * share + 1] = cut_last; }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) a.errs[blockIdx.x] = ctl[2];
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

// Joins the partial results of each sequence that a cut runs through. Block (cut, rows of a group, quarter of
// the channels) with `rpb` rows. A sequence with many parts takes the whole block to a row and quarter, each warp
// adding every NW-th part; one with few parts takes a warp to a row, all of its channels, in the blocks of the
// first quarter. The sums are added in a fixed order. One block more gathers the blocks' errors into the status word.
// It is a chain of reads that depend on one another, each of them the way to L2 and back (the cut, the parts' maxima and
// sums, the parts): what a read needs of the others is kept to that, and the first parts are on their way before
// their factors are known.
constexpr int kManyParts = 8;
template <int RG, int NW, int MINB>
__global__ void __launch_bounds__(32 * NW, MINB) latent_decode_join(DecodeArgs a, int rpb, int by_share)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cut = blockIdx.x / a.G, g = blockIdx.x % a.G, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (by_share ? blockIdx.x == gridDim.x - 1 : blockIdx.y == gridDim.y - 1) {       // the errors
        if ((by_share ? blockIdx.y : blockIdx.x) || blockIdx.z) return;
        int err = 0;
        for (int i = t; i < a.L * a.G; i += 32 * NW) err = max(err, a.errs[i]);
        err = __syncthreads_or(err == KDA_ERR_TIMEOUT) ? KDA_ERR_TIMEOUT : (__syncthreads_or(err) ? KDA_ERR_INVALID_ARG : 0);
        if (t == 0) *a.status = err;
        return;
    }
    // the share at whose end the cut-th cut sequence begins; with `by_share` (as many sequences as shares, or nearly)
    // block x looks at its own share instead of counting cuts
    __shared__ int s_cut[NW], s_found[3];
    __shared__ float4 s_o[NW][32];
    int share = cut, n = -1, last = -1;
    if (by_share) {
        const int2 x = reinterpret_cast<const int2 *>(a.meta)[share];
        n = x.x; last = x.y;
    } else {
        int before = 0;
        if (t == 0) s_found[1] = -1;
        for (int base = 0; base < a.L; base += 32 * NW) {
            const int i = base + t;
            const int2 x = i < a.L ? reinterpret_cast<const int2 *>(a.meta)[i] : make_int2(-1, -1);
            const bool is = x.x >= 0;
            const uint32_t ball = __ballot_sync(0xffffffffu, is);
            if (lane == 0) s_cut[warp] = __popc(ball);
            __syncthreads();
            int at = before + __popc(ball & ((1u << lane) - 1));
            for (int w = 0; w < NW; ++w) { if (w < warp) at += s_cut[w]; before += s_cut[w]; }
            if (is && at == cut) { s_found[0] = i; s_found[1] = x.x; s_found[2] = x.y; }
            __syncthreads();
        }
        share = s_found[0]; n = s_found[1]; last = s_found[2];
    }
    if (n < 0) return;
    const int parts = last - share + 1;
    const bool many = parts > kManyParts;
    if (!many && blockIdx.z > 0) return;
    const int quarters = 4 / gridDim.z;                        // of the channels, for this block, with many parts
    auto slot_of = [&](int s, int r) { return ((size_t)((share + s) * a.G + g) * 2 + (s == 0 ? 1 : 0)) * RG + r; };
    const int r_end = min(min(RG, a.Tq * a.H - g * RG), ((int)blockIdx.y + 1) * rpb);
    const size_t row0 = (size_t)n * a.Tq * a.H + g * RG;
    if (!many) {
        for (int r = blockIdx.y * rpb + warp; r < r_end; r += NW) {
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < parts) ml = *reinterpret_cast<const float2 *>(a.part_ml + slot_of(lane, r) * 2);
            const float m = warp_max(ml.x), f = ex2(ml.x - (m == -INFINITY ? 0.f : m));
            float l = f * ml.y;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            l = __shfl_sync(0xffffffffu, l, 0);
            float4 o[4] = {};
#pragma unroll 2
            for (int s = 0; s < parts; ++s) {
                const float fs = __shfl_sync(0xffffffffu, f, s);
                const float4 *src = reinterpret_cast<const float4 *>(a.part + slot_of(s, r) * kLatentDim) + lane;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 x = __ldcs(src + 32 * c);
                    o[c].x += fs * x.x; o[c].y += fs * x.y; o[c].z += fs * x.z; o[c].w += fs * x.w;
                }
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                reinterpret_cast<uint2 *>(a.out + (row0 + r) * kLatentDim)[32 * c + lane] =
                    make_uint2(pack_bf16x2(o[c].x * inv, o[c].y * inv), pack_bf16x2(o[c].z * inv, o[c].w * inv));
            if (lane == 0) a.lse[row0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
        return;
    }
    constexpr int PT = (kLanes + 32 * NW - 1) / (32 * NW);     // parts of a thread
    __shared__ float s_f[kLanes], s_red[2][NW];
    constexpr int EARLY = MINB == 1 ? 10 : 4;                                   // parts of a warp that are read before their factors are known
    for (int r = blockIdx.y * rpb; r < r_end; ++r) {
        float4 x[EARLY];
        auto part = [&](int s, int col) { return __ldcs(reinterpret_cast<const float4 *>(a.part + slot_of(s, r) * kLatentDim) + col); };
        auto early = [&](int col) {
#pragma unroll
            for (int i = 0; i < EARLY; ++i)
                if (warp + NW * i < parts) x[i] = part(warp + NW * i, col);
        };
        early(blockIdx.z * quarters * 32 + lane);
        float2 ml[PT];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            if (t + 32 * NW * i < parts) ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + slot_of(t + 32 * NW * i, r) * 2);
            m = fmaxf(m, ml[i].x);
        }
        m = warp_max(m);
        if (lane == 0) s_red[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) m = fmaxf(m, s_red[0][w]);
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            const float f = ex2(ml[i].x - (m == -INFINITY ? 0.f : m));
            l += f * ml[i].y;
            if (t + 32 * NW * i < parts) s_f[t + 32 * NW * i] = f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) s_red[1][warp] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) l += s_red[1][w];
        for (int qt = 0; qt < quarters; ++qt) {
            const int col = (blockIdx.z * quarters + qt) * 32 + lane;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (qt > 0) early(col);
#pragma unroll
            for (int i = 0; i < EARLY; ++i)
                if (warp + NW * i < parts) {
                    const float f = s_f[warp + NW * i];
                    o.x += f * x[i].x; o.y += f * x[i].y; o.z += f * x[i].z; o.w += f * x[i].w;
                }
#pragma unroll 4
            for (int s = warp + NW * EARLY; s < parts; s += NW) {
                const float f = s_f[s];
                const float4 y = part(s, col);
                o.x += f * y.x; o.y += f * y.y; o.z += f * y.z; o.w += f * y.w;
            }
            s_o[warp][lane] = o;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < NW; ++w) { const float4 x = s_o[w][lane]; o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w; }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                reinterpret_cast<uint2 *>(a.out + (row0 + r) * kLatentDim)[col] =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (col == 0) a.lse[row0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            }
            __syncthreads();
        }
    }
}

bool al(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Rows per group, groups and shares for Tq x H query rows.
struct Plan { int RG, G, L; size_t meta, errs, part, ml, total; };
Plan plan_of(long long rows)
{
    Plan p;
    p.RG = rows <= 32 ? 32 : 64;
    p.G = (int)((rows + p.RG - 1) / p.RG);
    p.L = p.G >= kLanes ? 1 : kLanes / p.G;
    size_t off = kStatusBytes;
    p.meta = off; off += align256((size_t)p.L * 8);
    p.errs = off; off += align256((size_t)p.L * p.G * 4);
    p.ml = off; off += align256((size_t)p.L * p.G * 2 * p.RG * 8);
    p.part = off; off += (size_t)p.L * p.G * 2 * p.RG * kLatentDim * 4;
    p.total = off;
    return p;
}

template <int RG>
cudaError_t launch(const DecodeArgs &a, const CUtensorMap &tq, const CUtensorMap &tc, cudaStream_t st)
{
    auto kern = latent_decode_kernel<RG>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<RG>::TOTAL);
    if (e != cudaSuccess) return e;
    if ((e = launch_after(kern, a.L * a.G, Lay<RG>::NT, Lay<RG>::TOTAL, st, a, tq, tc)) != cudaSuccess) return e;
    // the join's blocks may be scheduled while the last shares finish; they wait for the whole first kernel
    // at most one cut a share and one a sequence; with few of them a block per row and quarter, else four rows to a block
    const int by_share = 2 * a.N >= a.L, cuts = by_share ? a.L : a.N, rows = RG < a.Tq * a.H ? RG : a.Tq * a.H;
    const int rpb = cuts * a.G <= 8 ? 1 : 4;
    const dim3 grid(cuts * a.G + (by_share ? 1 : 0), (rows + rpb - 1) / rpb + (by_share ? 0 : 1), by_share ? 1 : 4);
    // with a block to an SM at most, ten parts a warp are read early (one sequence of 128K tokens, 32 heads: 43.2 us with
    // none, 40.3 so); with more blocks, four, so that two fit
    if (by_share) return launch_after(latent_decode_join<RG, 4, 8>, grid, 128, 0, st, a, rpb, by_share);
    if (cuts * a.G * ((rows + rpb - 1) / rpb) * 4 <= kLanes) return launch_after(latent_decode_join<RG, 16, 1>, grid, 512, 0, st, a, rpb, by_share);
    return launch_after(latent_decode_join<RG, 16, 2>, grid, 512, 0, st, a, rpb, by_share);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_latent_decode_workspace_size(int N, int Tq, int H)
{
    if (N < 0 || Tq < 1 || H < 1 || (long long)Tq * H > 65536) return 0;
    return plan_of((long long)Tq * H).total;
}

kda_status_t kda_latent_decode_step(const void *q, const void *cache, const int32_t *page_table, const int32_t *seq_lens,
                                    void *out, float *lse, int N, int Tq, int H, int dc, int dr, int page_size,
                                    long long num_pages, int max_pages, float scale, kda_dtype_t dtype, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (N < 0 || Tq < 1 || H < 1 || page_size < 1 || num_pages < 0 || max_pages < 0) return KDA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 || dc != kLatentDim || (dr != 0 && dr != kSharedDim) || page_size % 16 != 0) return KDA_ERR_UNSUPPORTED;
    if (num_pages * page_size > 0x7fff0000LL || (long long)max_pages * page_size > 0x7fff0000LL ||
        (long long)N * ((long long)max_pages * page_size / KT + 1) > 0x7fffffffLL || (long long)Tq * H > 65536 || (long long)N * Tq * H > 0x7fff0000LL || N > kMaxGridDim)
        return KDA_ERR_UNSUPPORTED;
    if (!workspace || !al(workspace, 16) || workspace_bytes < kda_latent_decode_workspace_size(N, Tq, H)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 0) return cudaMemsetAsync(workspace, 0, kStatusBytes, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    if (!q || !seq_lens || !out || !lse) return KDA_ERR_INVALID_ARG;
    if (!al(q, 16) || !al(cache, 16) || !al(page_table, 4) || !al(seq_lens, 4) || !al(out, 16) || !al(lse, 4))
        return KDA_ERR_INVALID_ARG;
    if (max_pages > 0 && (!page_table || (num_pages > 0 && !cache))) return KDA_ERR_INVALID_ARG;
    const Plan pl = plan_of((long long)Tq * H);
    unsigned char *ws = (unsigned char *)workspace;
    DecodeArgs a;
    a.table = page_table; a.lens = seq_lens; a.out = (__nv_bfloat16 *)out; a.lse = lse;
    a.N = N; a.Tq = Tq; a.H = H; a.R = dr; a.page = page_size; a.pages = (int)num_pages; a.max_pages = max_pages;
    a.box = KT;
    while (page_size % a.box) a.box >>= 1;                     // 64, 32 or 16
    a.G = pl.G; a.L = pl.L; a.scale_log2 = scale * 1.44269504088896341f;
    a.meta = (int32_t *)(ws + pl.meta); a.errs = (int32_t *)(ws + pl.errs);
    a.part_ml = (float *)(ws + pl.ml); a.part = (float *)(ws + pl.part);
    a.status = (int32_t *)ws;
    const long long W = kLatentDim + dr, qrows = (long long)N * Tq * H, crows = num_pages * page_size;
    // without a cache row every length is idle (or refused on the device), and no copy is made
    CUtensorMap tq = {}, tc = {};
    if (crows > 0 && (!bf16_rows_map(&tq, q, W, qrows, W, 64, pl.RG) || !bf16_rows_map(&tc, cache, W, crows, W, 64, a.box)))
        return KDA_ERR_CUDA;
    if (crows == 0) a.max_pages = 0;
    const cudaError_t e = pl.RG == 32 ? launch<32>(a, tq, tc, st) : launch<64>(a, tq, tc, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
