// kvq_attn_e2m1_tc.cu -- split-K paged attention over the 4-bit (E2M1) cache for
// many query rows per kv head (MTP verify: G heads x q_len rows, 16 < rows <= 64,
// head_dim 128, no top-k list) on the fifth-generation tensor cores.
//
// The same partials as attn_e2m1_kernel, which decodes every code once per
// 8-row n-tile group and multiplies with mma.sync: at 32 rows it is bound by
// those multiplies and their registers.  Here a code is decoded once, by the
// warp that fetched it, into the operand of an M = 128 MMA.
//
// One CTA per (split, kv head, sequence), two CTAs per SM (up to 32 rows), tiles
// of 128 tokens (32 pages), token 32 d + l in lane l of quadrant d:
//  * warps 4-7 (decode): fetch the raw pages of their 32 tokens (cp.async, K and
//    V apart, the next tile's as soon as this one's are in registers) and write
//    K = code * block scale (exact fp16) to tensor memory -- the A operand of
//    S^T = K Q^T -- and V to shared memory, MN-major -- the A operand of
//    O^T = V^T P^T.  K and V are double-buffered.
//  * warp 12 issues the MMAs, S^T of tile t + 1 before P V of tile t.
//  * warps 0-3 and 8-11 (softmax): thread = token and half of the rows (with all
//    32 rows in one thread the softmax was a tile's longest chain: 153 -> 143 us);
//    a row's reference moves only when a score rises more than 2^8 above it,
//    decided by one OR-reduction of a half's four warps a tile; P^T (fp16) to
//    shared memory; row sums in registers.
// 64 sequences of 1K to 32K, 4 kv heads, 32 rows, 4 splits: 137.5 us, 2.4 TB/s of
// pages, a tile in 1.1 us on an SM's two CTAs (the mma.sync kernel: 210 us).  A tile
// takes 4700 warp instructions: 56 % of the issue slots and 44 % of the ALU are busy,
// the tensor cores 12 %, DRAM 31 %.  What bounds it is the decode warps' chain over a
// tile (about 2400 cycles alone on an SM, of which the two conversions take 900 and the
// reads of the raw pages with the next copies' issue 900), and two CTAs per SM to hide
// it.  Measured and rejected: a bulk copy a page in place of the 16-byte pieces (143 ->
// 164 us), the copies issued between the blocks of the conversion (143 -> 155 us),
// K and V decoded by four warps each (17 warps of 56 registers: 137.5 -> 157 us).
// Every wait is bounded (about 2 s): on expiry the CTA reports
// KVQ_DEV_TIMEOUT, lets its copies and MMAs drain, gives its rows zero weight
// and frees its tensor memory.
#include <cfloat>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_attn_kernel.cuh"
#include "kvq_e2m1.cuh"
#include "kvq_tcgen05.cuh"
#include "kvq_warp.cuh"

namespace kvq {

namespace {

constexpr int kVtD = 128;
constexpr int kVtTile = 128;                       // tokens per tile
constexpr int kVtPages = kVtTile / 4;
constexpr int kVtDecode = 4, kVtMma = 12;          // first decode warp, the MMA warp; the others do the softmax
constexpr int kVtThreads = 32 * 13;
constexpr int kVtPage = e2m1_page_bytes(kVtD);     // 288
constexpr int kVtRaw = 8 * kVtPage;                // a decode warp's raw K (or V) of one tile
constexpr float kNoRef = -1e30f;                   // reference of a row that has seen no token

template <int NR>
struct VtLayout {
    static constexpr int kV = 0;                                  // [2] V^T: 128 ch x 128 tok fp16, MN-major
    static constexpr int kQ = kV + 2 * kVtTile * kVtD * 2;        // Q: NR x 128 fp16, K-major
    static constexpr int kP = kQ + NR * 256;                      // [2] P^T: NR x 128 tok fp16, MN-major
    static constexpr int kRaw = kP + 2 * NR * 256;                // [4 warps][K, V] raw pages
    static constexpr int kNref = kRaw + 4 * 2 * kVtRaw;           // [4 warps][NR] float: minus the reference
    static constexpr int kCorr = kNref + 4 * NR * 4;              // [4 warps][NR] float
    static constexpr int kWmax = kCorr + 4 * NR * 4;              // [4 warps][NR] float: maxima, then sums
    static constexpr int kBar = kWmax + 4 * NR * 4;
    // barriers: k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], drain
    static constexpr int kNumBars = 13;
    static constexpr int kAbort = kBar + 8 * kNumBars;
    static constexpr int kTmemSlot = kAbort + 8;
    static constexpr int kBytes = kTmemSlot + 8;
    // tensor-memory columns: K [2] (64: 128 fp16 per lane), S^T [2], O^T
    static constexpr int kColK = 0, kColS = 128, kColO = 128 + 2 * NR;
    static constexpr int kCols = 128 + 3 * NR <= 256 ? 256 : 512;
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int PENDING>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Named barriers 1 and 2 of 128 threads, one for each half of the softmax warps (with the number an
// immediate: a barrier number in a register reserves all sixteen).  The first also ORs `x`.
template <int ID>
__device__ __forceinline__ bool bar_or_id(bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                 "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "n"(ID), "r"(x ? 1u : 0u) : "memory");
    return r != 0;
}

__device__ __forceinline__ bool half_or(int half, bool x) { return half ? bar_or_id<2>(x) : bar_or_id<1>(x); }

__device__ __forceinline__ void half_sync(int half)
{
    if (half) asm volatile("bar.sync 2, 128;" ::: "memory");
    else asm volatile("bar.sync 1, 128;" ::: "memory");
}

// one row's 128 codes (16 words) times their block scales, as fp16 pairs of adjacent
// channels; sc: the page's scale words [8 blocks], sel picks this token's byte twice
template <typename Emit>
__device__ __forceinline__ void decode_row(const uint4 (&x)[4], const uint4 (&sc)[2], uint32_t sel, bool live, Emit emit)
{
    const uint32_t xw[16] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w,
                             x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w};
    const uint32_t sw[8] = {sc[0].x, sc[0].y, sc[0].z, sc[0].w, sc[1].x, sc[1].y, sc[1].z, sc[1].w};
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint32_t s = live ? cvt_lo(__byte_perm(sw[b], 0u, sel)) : 0u;
        uint32_t w[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[4 * u + 0] = hmul2(e2m1_pair<0>(xw[2 * b + u]), s);
            w[4 * u + 1] = hmul2(e2m1_pair<1>(xw[2 * b + u]), s);
            w[4 * u + 2] = hmul2(e2m1_pair<2>(xw[2 * b + u]), s);
            w[4 * u + 3] = hmul2(e2m1_pair<3>(xw[2 * b + u]), s);
        }
        emit(b, w);
    }
}

// lane r of the warp ends with the maximum (or sum) over the warp's 32 lanes of v[r]
template <bool MAX>
__device__ __forceinline__ float across_lanes(float (&v)[32], int lane)
{
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) {
        const bool hi = (lane & k) != 0;
#pragma unroll
        for (int i = 0; i < k; ++i) {
            const float send = hi ? v[i] : v[i + k], keep = hi ? v[i + k] : v[i];
            const float recv = __shfl_xor_sync(kFull, send, k);
            v[i] = MAX ? fmaxf(keep, recv) : keep + recv;
        }
    }
    return v[0];
}

}  // namespace

template <int NR>
__global__ void __launch_bounds__(kVtThreads, NR <= 32 ? 2 : 1) attn_e2m1_tc_kernel(const AttnArgs a)
{
    using T = VtLayout<NR>;
    static_assert(NR == 32 || NR == 64, "a half has 16 or 32 rows");
    constexpr int D = kVtD;
    extern __shared__ __align__(128) uint8_t smem[];
    const int s = blockIdx.x, g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = smem_u32(smem + T::kBar);
    auto k_full = [&](int x) { return bar + 8 * x; };
    auto k_empty = [&](int x) { return bar + 16 + 8 * x; };
    auto v_full = [&](int x) { return bar + 32 + 8 * x; };
    auto v_empty = [&](int x) { return bar + 48 + 8 * x; };
    auto s_full = [&](int x) { return bar + 64 + 8 * x; };
    auto p_full = [&](int x) { return bar + 80 + 8 * x; };
    const uint32_t b_drain = bar + 96;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + T::kAbort);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + T::kTmemSlot);

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(k_full(x), 4);
            mbar_init(k_empty(x), 1);
            mbar_init(v_full(x), 4);
            mbar_init(v_empty(x), 1);
            mbar_init(s_full(x), 1);
            mbar_init(p_full(x), 8);
        }
        mbar_init(b_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kVtMma) tmem_alloc(smem_u32(tmem_slot), T::kCols);
    grid_dependency_wait();   // inputs may come from the previous kernel (e.g. the append)
    // sequences longest first: the lengths of a verify batch vary over a grid of several waves
    SeqPick pick = seq_identity(a, blockIdx.z);
    const bool keep_order = lpt_classify(a, smem, T::kQ);
    tc_fence_before();
    if (!__syncthreads_and(keep_order)) pick = lpt_pick(a, blockIdx.z, smem);
    tc_fence_after();
    const int b = pick.b;
    const SplitRange sr = split_range(a, s, b, pick.L, 0);
    const int L = sr.L, item0 = sr.item0, item1 = sr.item1;
    const int ntiles = (item1 - item0 + kVtPages - 1) / kVtPages;
    if (threadIdx.x == 0 && !sr.len_ok) report(a.err_flag, KVQ_DEV_BAD_LEN);
    // Q rows (padding rows zero) into the K-major Q tile: element (r, d) at
    // (r/8) * 2048 + (d/8) * 128 + (r%8) * 16 + (d%8) * 2
    for (int idx = threadIdx.x; idx < NR * (D / 8); idx += kVtThreads) {
        const int r = (idx & 7) + 8 * (idx / (8 * (D / 8))), c = (idx / 8) % (D / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < a.rows) {
            const int i = r / a.group, h = g * a.group + r % a.group;
            v = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(a.q) +
                                                 (((int64_t)b * a.q_len + i) * a.num_q_heads + h) * D + 8 * c);
        }
        *reinterpret_cast<uint4 *>(smem + T::kQ + (r >> 3) * 2048 + c * 128 + (r & 7) * 16) = v;
    }
    fence_async_smem();
    __syncthreads();
    launch_dependents();      // this CTA holds its tensor memory already
    const uint32_t tmem = *tmem_slot;

    if (warp == kVtMma) {
        // ================= MMA issue =================
        // The whole warp walks the tiles and one elected lane issues: addresses and descriptors then stay
        // warp-uniform, and an MMA costs its 17 (A in tensor memory) or 41 cycles (A in shared memory) instead
        // of about 46 to 85 from a branch on the lane.
        if (ntiles > 0) {
            const bool one = elect_one();
            const uint32_t id_qk = umma_idesc_f16(kVtTile, NR, false, false);
            const uint32_t id_pv = umma_idesc_f16(kVtTile, NR, true, true);
            const uint64_t dq = umma_desc(smem_u32(smem + T::kQ), 128, (D / 8) * 128);
            const uint64_t dv0 = umma_desc(smem_u32(smem + T::kV), (D / 8) * 128, 128);
            const uint64_t dp = umma_desc(smem_u32(smem + T::kP), NR * 16, 128);
            // S^T[tok][row] = sum_d K[tok][d] Q[row][d]
            auto scores = [&](int t) {
                const int x = t & 1;
                if (!mbar_wait_warp(k_full(x), (t >> 1) & 1, abort_flag, a.err_flag)) return false;
                tc_fence_after();
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        umma_tmem_a(tmem + T::kColS + x * NR, tmem + T::kColK + x * 64 + ks * 8, dq + (uint64_t)(ks * 16), id_qk,
                                    ks > 0);
                    umma_commit(s_full(x));
                    umma_commit(k_empty(x));
                }
                __syncwarp();
                return true;
            };
            bool ok = scores(0);
            for (int t = 0; ok && t < ntiles; ++t) {
                const int x = t & 1;
                if (t + 1 < ntiles && !scores(t + 1)) break;
                if (!mbar_wait_warp(v_full(x), (t >> 1) & 1, abort_flag, a.err_flag)) break;
                if (!mbar_wait_warp(p_full(x), (t >> 1) & 1, abort_flag, a.err_flag)) break;
                tc_fence_after();
                // O^T[ch][row] += sum_tok V[tok][ch] P[tok][row], both MN-major
                const uint64_t dv = dv0 + (uint64_t)(x * (kVtTile * D * 2 / 16)), dpx = dp + (uint64_t)(x * NR * 16);
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < kVtTile / 16; ++ks)
                        umma_smem_a(tmem + T::kColO, dv + (uint64_t)(ks * 2 * (D / 8) * 8), dpx + (uint64_t)(ks * 2 * NR), id_pv,
                                    t > 0 || ks > 0);
                    umma_commit(v_empty(x));
                }
                __syncwarp();
            }
            // every MMA issued so far completes before the tensor memory is freed
            if (one) umma_commit(b_drain);
            mbar_wait_bounded(b_drain, 0, nullptr, a.err_flag, 100000000ull);
        }
        __syncwarp();
    } else if (warp >= kVtDecode && warp < kVtDecode + 4) {
        // ================= decode warps =================
        const int d = warp - kVtDecode;
        const uint32_t lane_base = (uint32_t)(32 * d) << 16;
        const uint8_t *rawk = smem + T::kRaw + d * 2 * kVtRaw, *rawv = rawk + kVtRaw;
        const uint32_t rawk_s = smem_u32(rawk), rawv_s = smem_u32(rawv);
        const int64_t page_stride = (int64_t)a.num_kv_heads * kVtPage;
        const uint8_t *kpool = static_cast<const uint8_t *>(a.k_cache) + (int64_t)g * kVtPage;
        const uint8_t *vpool = static_cast<const uint8_t *>(a.v_cache) + (int64_t)g * kVtPage;
        // pages of this warp in tile t, lane l (mod 8) holding page l's number: -1 past the split's end
        auto raw_page = [&](int t) {
            const int it = item0 + t * kVtPages + 8 * d + (lane & 7);
            return it < item1 ? __ldg(sr.bt_row + it) : -1;
        };
        const unsigned num_pages = (unsigned)min(a.num_pages, (int64_t)0x80000000ll);
        auto checked = [&](int phys, int t) {
            if (__builtin_expect((unsigned)phys < num_pages, 1)) return phys;
            if (item0 + t * kVtPages + 8 * d + (lane & 7) < item1 && lane < 8) report(a.err_flag, KVQ_DEV_BAD_PAGE);
            return -1;
        };
        // 8 pages as 144 pieces of 16 bytes, consecutive lanes on consecutive pieces; missing
        // pages are read from page 0 (whatever it holds) and masked
        int piece[5];                       // the page of this lane's i-th piece
        auto pieces = [&](int phys) {
            const int have = max(phys, 0);
#pragma unroll
            for (int i = 0; i < 5; ++i) piece[i] = __shfl_sync(kFull, have, (((i * 32 + lane) * 57) >> 10) & 7);
        };
        auto fetch = [&](const uint8_t *pool, uint32_t dst) {
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int c = i * 32 + lane, p = (c * 57) >> 10;   // c / 18 for c < 144
                if (c < 8 * (kVtPage / 16)) copy16(dst + c * 16, pool + piece[i] * page_stride + (c * 16 - p * kVtPage));
            }
            commit_copies();
        };
        int cur = -1, nxt = raw_page(1);
        if (ntiles > 0) {
            cur = checked(raw_page(0), 0);
            pieces(cur);
            fetch(kpool, rawk_s);
            fetch(vpool, rawv_s);
        }
        const int row_off = (lane >> 2) * kVtPage + (lane & 3) * (D / 2), scale_off = (lane >> 2) * kVtPage + 2 * D;
        const uint32_t sel = 0x11u * (lane & 3);            // this token's byte of a scale word, twice
        const int tt = 32 * d + lane;
        bool ok = true;
        for (int t = 0; t < ntiles; ++t) {
            const int x = t & 1;
            const bool more = t + 1 < ntiles;
            const int ahead = raw_page(t + 2);
            if (more) nxt = checked(nxt, t + 1);
            pieces(nxt);
            // this warp's tokens of the tile: inside a page that exists, below L
            const int pos = (item0 + t * kVtPages + 8 * d) * 4 + lane;
            const bool live = __shfl_sync(kFull, cur, lane >> 2) >= 0 && pos < L;
            // ---- K ----
            wait_copies<1>();
            __syncwarp();
            uint4 raw[4], sc[2];
#pragma unroll
            for (int u = 0; u < 4; ++u) raw[u] = *reinterpret_cast<const uint4 *>(rawk + row_off + 16 * u);
#pragma unroll
            for (int u = 0; u < 2; ++u) sc[u] = *reinterpret_cast<const uint4 *>(rawk + scale_off + 16 * u);
            __syncwarp();
            if (more) fetch(kpool, rawk_s);
            else commit_copies();
            if (t >= 2 && !mbar_wait_warp(k_empty(x), ((t >> 1) - 1) & 1, abort_flag, a.err_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            {
                uint32_t w16[16];
                decode_row(raw, sc, sel, true, [&](int blk, const uint32_t(&w)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w16[8 * (blk & 1) + e] = w[e];
                    if (blk & 1) tmem_st16(tmem + lane_base + T::kColK + x * 64 + 16 * (blk >> 1), w16);
                });
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(k_full(x));
            // ---- V: (ch, tok) at (tok/8) * 2048 + (ch/8) * 128 + (tok%8) * 16; a slot without a token is
            // zero: its bits may be NaN, and P = 0 alone leaves 0 * NaN ----
            wait_copies<1>();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 4; ++u) raw[u] = *reinterpret_cast<const uint4 *>(rawv + row_off + 16 * u);
#pragma unroll
            for (int u = 0; u < 2; ++u) sc[u] = *reinterpret_cast<const uint4 *>(rawv + scale_off + 16 * u);
            __syncwarp();
            if (more) fetch(vpool, rawv_s);
            else commit_copies();
            if (t >= 2 && !mbar_wait_warp(v_empty(x), ((t >> 1) - 1) & 1, abort_flag, a.err_flag)) {
                ok = false;
                break;
            }
            {
                uint8_t *dst = smem + T::kV + x * kVtTile * D * 2 + (tt >> 3) * ((D / 8) * 128) + (tt & 7) * 16;
                decode_row(raw, sc, sel, live, [&](int blk, const uint32_t(&w)[8]) {
                    *reinterpret_cast<uint4 *>(dst + (2 * blk) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(dst + (2 * blk + 1) * 128) = make_uint4(w[4], w[5], w[6], w[7]);
                });
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_full(x));
            cur = nxt;
            nxt = ahead;
        }
        (void)ok;
        wait_copies<0>();
    } else {
        // ================= softmax warps: thread = token and half of the rows =================
        constexpr int NH2 = NR / 2;                  // rows of a half
        const int q = warp & 3, half = warp >> 3, r0 = half * NH2;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int tt = 32 * q + lane;
        const int win0 = L - a.q_len;                // row i of the window sees positions <= win0 + i
        float *nref = reinterpret_cast<float *>(smem + T::kNref) + q * NR + r0;   // from this half's first row on
        float *corr = reinterpret_cast<float *>(smem + T::kCorr) + q * NR + r0;
        float *wmax = reinterpret_cast<float *>(smem + T::kWmax) + r0;
        const float qk = a.qk_scale_log2;
        const float2 qk2 = make_float2(qk, qk);
        if (lane < NH2) nref[lane] = -kNoRef;
        __syncwarp();
        float2 l2[NH2 / 2];                           // this thread's sums of P, by row
#pragma unroll
        for (int r = 0; r < NH2 / 2; ++r) l2[r] = make_float2(0.f, 0.f);
        // the page of this thread's token (-1: past the split's end); the decode warps report bad ones
        const unsigned num_pages = (unsigned)min(a.num_pages, (int64_t)0x80000000ll);
        auto token_page = [&](int t) {
            const int it = item0 + t * kVtPages + 8 * q + (lane >> 2);
            return it < item1 ? __ldg(sr.bt_row + it) : -1;
        };
        int page = token_page(0);
        bool ok = true;
#ifdef KVQ_TEST_STALL_SOFTMAX
        // Test builds only (never the library's default build): a wait, bounded by KVQ_TEST_STALL_SOFTMAX
        // nanoseconds, for the first P V, which needs the P of these warps: it always gives up.
        ok = __all_sync(kFull, mbar_wait_bounded(v_empty(0), 0, abort_flag, a.err_flag, KVQ_TEST_STALL_SOFTMAX));
#endif
        for (int t = 0; t < ntiles; ++t) {
            const int x = t & 1;
            const unsigned have = __ballot_sync(kFull, (unsigned)page < num_pages);   // tokens with a page
            page = token_page(t + 1);
            ok = ok && mbar_wait_warp(s_full(x), (t >> 1) & 1, abort_flag, a.err_flag);
            tc_fence_after();
            float2 z[NH2 / 2];
            {
                uint32_t r16[NH2 / 16][16];
#pragma unroll
                for (int c = 0; c < NH2 / 16; ++c) tmem_ld16(tmem + lane_base + T::kColS + x * NR + r0 + 16 * c, r16[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < NH2 / 16; ++c) {
                    tmem_regs_ready(r16[c]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[8 * c + e] = make_float2(__uint_as_float(r16[c][2 * e]), __uint_as_float(r16[c][2 * e + 1]));
                }
            }
            // rows of window row i see positions <= win0 + i; tokens without a page none
            const int pos = (item0 + t * kVtPages) * 4 + tt;
            if (have != kFull || (item0 + (t + 1) * kVtPages) > (win0 + 1) / 4) {
                const int first = !((have >> lane) & 1u) ? NR : pos > win0 ? a.group * (pos - win0) : 0;
#pragma unroll
                for (int r = 0; r < NH2 / 2; ++r) {
                    if (r0 + 2 * r < first) z[r].x = -INFINITY;
                    if (r0 + 2 * r + 1 < first) z[r].y = -INFINITY;
                }
            }
            // z = score - reference (log2 units)
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < NH2 / 2; r += 2) {
                const float4 nr = *reinterpret_cast<const float4 *>(nref + 2 * r);
                z[r] = ffma2(z[r], qk2, make_float2(nr.x, nr.y));
                z[r + 1] = ffma2(z[r + 1], qk2, make_float2(nr.z, nr.w));
                m4[(r / 2) & 3] = fmax3(fmax3(m4[(r / 2) & 3], z[r].x, z[r].y), z[r + 1].x, z[r + 1].y);
            }
            const bool above = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) > 8.f;
            if (__builtin_expect(half_or(half, above || !ok), 0)) {
                // rare: exact maxima of the tile's rows, references that rose by more than 2^8, O and the sums rescaled
                if (half_or(half, !ok)) {     // some warp gave up: all four leave together
                    ok = false;
                    break;
                }
                // the scores themselves again (z of a row without a reference has lost them)
                auto reload = [&](bool absolute) {
#pragma unroll
                    for (int c = 0; c < NH2; c += 16) {
                        uint32_t r16[16];
                        tmem_ld16(tmem + lane_base + T::kColS + x * NR + r0 + c, r16);
                        tmem_wait_ld();
                        tmem_regs_ready(r16);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = c / 2 + e;
                            const bool dead_x = z[r].x == -INFINITY, dead_y = z[r].y == -INFINITY;
                            const float2 n = absolute ? make_float2(0.f, 0.f) : make_float2(nref[2 * r], nref[2 * r + 1]);
                            z[r] = ffma2(make_float2(__uint_as_float(r16[2 * e]), __uint_as_float(r16[2 * e + 1])), qk2, n);
                            if (dead_x) z[r].x = -INFINITY;
                            if (dead_y) z[r].y = -INFINITY;
                        }
                    }
                };
                reload(true);
                {
                    float v[32];
#pragma unroll
                    for (int r = 0; r < 32; ++r)
                        v[r] = r < NH2 ? ((r & 1) ? z[r / 2 % (NH2 / 2)].y : z[r / 2 % (NH2 / 2)].x) : -INFINITY;
                    const float m = across_lanes<true>(v, lane);
                    if (lane < NH2) wmax[q * NR + lane] = m;
                }
                half_sync(half);
                if (lane < NH2) {
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < 4; ++w) m = fmaxf(m, wmax[w * NR + lane]);
                    const float old = -nref[lane];
                    const bool move = m > old + 8.f;
                    corr[lane] = move ? fast_exp2(old - m) : 1.f;   // 0 where there was no reference
                    if (move) nref[lane] = -m;
                }
                __syncwarp();
                reload(false);
#pragma unroll
                for (int r = 0; r < NH2 / 2; ++r) {
                    l2[r].x *= corr[2 * r];
                    l2[r].y *= corr[2 * r + 1];
                }
                if (t > 0) ok = ok && mbar_wait_warp(v_empty((t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag, a.err_flag);
                tc_fence_after();
                if (t > 0) {
#pragma unroll
                    for (int c = 0; c < NH2; c += 16) {
                        uint32_t r16[16];
                        tmem_ld16(tmem + lane_base + T::kColO + r0 + c, r16);
                        tmem_wait_ld();
                        tmem_regs_ready(r16);
#pragma unroll
                        for (int e = 0; e < 16; ++e) r16[e] = __float_as_uint(__uint_as_float(r16[e]) * corr[c + e]);
                        tmem_st16(tmem + lane_base + T::kColO + r0 + c, r16);
                    }
                    tmem_wait_st();
                }
                half_sync(half);              // the maxima have been read
            }
            // P = 2^z; P^T: (row, tok) at (tok/8) * NR*16 + (row/8) * 128 + (tok%8) * 16, once the P V of two tiles
            // ago has read the buffer
            if (t > 1) ok = ok && mbar_wait_warp(v_empty(x), ((t >> 1) - 1) & 1, abort_flag, a.err_flag);
            uint8_t *dst = smem + T::kP + x * NR * 256 + (tt >> 3) * (NR * 16) + (tt & 7) * 16;
#pragma unroll
            for (int c = 0; c < NH2 / 8; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = make_float2(fast_exp2(z[4 * c + e].x), fast_exp2(z[4 * c + e].y));
                    l2[4 * c + e] = fadd2(l2[4 * c + e], p);
                    w[e] = pack_half2(p.x, p.y);
                }
                *reinterpret_cast<uint4 *>(dst + (r0 / 8 + c) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(p_full(x));
        }
        // ---- epilogue: row sums over the four warps, then O^T / l ----
        {
            float v[32];
#pragma unroll
            for (int r = 0; r < 32; ++r) v[r] = r < NH2 ? ((r & 1) ? l2[r / 2 % (NH2 / 2)].y : l2[r / 2 % (NH2 / 2)].x) : 0.f;
            const float l = across_lanes<false>(v, lane);
            if (lane < NH2) wmax[q * NR + lane] = l;
        }
        if (ok && ntiles > 0)
            ok = mbar_wait_warp(v_empty((ntiles - 1) & 1), ((ntiles - 1) >> 1) & 1, abort_flag, a.err_flag);
        if (!half_or(half, !ok)) {
            tc_fence_after();
            const int S = a.num_splits;
            int unit_l = -1;                         // lane r: the workspace unit of this half's row r, -1 for a padding row
            float coef_l = 0.f;
            if (lane < NH2 && r0 + lane < a.rows) {
                const int r = r0 + lane;
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) l += wmax[w * NR + lane];
                const int i = r / a.group, hh = g * a.group + r % a.group;
                unit_l = ((b * a.num_q_heads + hh) * a.q_len + i) * S + s;
                const bool nan = l != l;             // a NaN score: the split outweighs every other in the combine
                coef_l = l == 0.f ? 0.f : a.out_scale / l;
                if (q == 0) {
                    a.ws_m[unit_l] = nan ? FLT_MAX : l > 0.f ? -nref[lane] * kLn2 : -INFINITY;
                    a.ws_l[unit_l] = nan ? 1.f : l;
                }
            }
            if (ntiles > 0) {
#pragma unroll
                for (int c = 0; c < NH2; c += 16) {
                    uint32_t r16[16];
                    tmem_ld16(tmem + lane_base + T::kColO + r0 + c, r16);
                    tmem_wait_ld();
                    tmem_regs_ready(r16);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int unit = __shfl_sync(kFull, unit_l, c + e);
                        const float k = __shfl_sync(kFull, coef_l, c + e);
                        if (unit >= 0 && k != 0.f) a.ws_o[(int64_t)unit * D + tt] = __uint_as_float(r16[e]) * k;
                    }
                }
            }
        }
    }

    // ---- teardown: copies landed (each decode warp waited), MMAs complete, tensor memory freed ----
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        for (int r = threadIdx.x; r < a.rows; r += kVtThreads) {
            const int i = r / a.group, hh = g * a.group + r % a.group;
            const int64_t unit = (((int64_t)b * a.num_q_heads + hh) * a.q_len + i) * a.num_splits + s;
            a.ws_m[unit] = -INFINITY;
            a.ws_l[unit] = 0.f;
        }
    }
    tc_fence_after();
    __syncthreads();
    if (warp == kVtMma) tmem_dealloc(tmem, T::kCols);
}

template <int NR>
static cudaError_t launch_vt(const AttnArgs &a, cudaStream_t stream)
{
    constexpr int bytes = VtLayout<NR>::kBytes;
    static uint64_t configured = 0;   // one bit per device ordinal
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
        e = cudaFuncSetAttribute(attn_e2m1_tc_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    return launch_pdl(attn_e2m1_tc_kernel<NR>, dim3(a.num_splits, a.num_kv_heads, a.batch), dim3(kVtThreads), bytes, stream, a);
}

cudaError_t launch_attention_e2m1_tc(const AttnArgs &a, cudaStream_t stream)
{
    if (a.rows <= 32) return launch_vt<32>(a, stream);
    return launch_vt<64>(a, stream);
}

}  // namespace kvq
