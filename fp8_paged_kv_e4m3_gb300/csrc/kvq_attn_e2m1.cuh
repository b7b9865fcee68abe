// kvq_attn_e2m1.cuh -- split-K paged decode / verify attention over the 4-bit
// (E2M1) cache.
//
// The attention is the split kernel's: s_j = sm_scale k_scale sum_d q_d K_jd,
// out = v_scale sum_j p_j V_j / sum_j p_j with K, V = E2M1(code) * b, an exact
// fp16 value (at most 6 significant bits, magnitude at most 2688), so both
// products run on fp16 tensor-core instructions (mma.sync m16n8k16, tokens on
// M, query rows on N) with binary32 sums and the layer scales hoisted.
//
// One CTA of W warps per (split, kv head, sequence); a warp takes units of 32
// tokens (two tiles of four pages) and keeps its own softmax.  Units come
// through a ring of the warp's own in shared memory, copied ahead by cp.async:
// a lane copies exactly the bytes of its own matrix fragments and reads them
// back itself, so no lane and no warp waits for another until the merge:
//   rows of a K tile   tile row r < 8 is token r % 2 of page r / 2, row r + 8
//                      its token 2 + r % 2.  Lane (gid, t) holds the D / 4
//                      channels from t D / 4 on of both rows, and their scales.
//   columns of P V     k index 2t, 2t + 1 are tokens 0, 1 and 2t + 8, 2t + 9
//                      tokens 2, 3 of page t: lane (gid, t) holds the D / 8
//                      channels from gid D / 8 on of all four tokens.  Two
//                      tokens' codes are interleaved nibble by nibble, so that
//                      one conversion gives one channel of both.
// The order of channels and tokens inside a product is free as long as both
// operands share it: Q is loaded, and O stored, in this order.
//
// What bounds it.  A cached element is 0.5625 bytes, half an E4M3 one, but costs
// the same conversion, scaling and product, so where the E4M3 kernel waits for
// memory this one also fills the ALU: a token's K and V (256 channels) take 128
// conversions and 128 products by block scales, 16 lanes a clock and scheduler
// each.  8 query rows a kv head, 4 kv heads, head_dim 128: B 4 x 262144 tokens
// 111 us (5.45 TB/s, 80 % of the copy peak; ALU 50 % and issue slots 58 % busy);
// B 32 x 32768 116 us (77 %); B 32 x 4096 20.6 us (54 %: one wave, of which the
// first pages' arrival and the merge take about 5 us).  With 16 rows 51 us at
// B 32 x 8192 (3.0 TB/s).
#pragma once

#include <cfloat>

#include "kvq_attn_kernel.cuh"
#include "kvq_e2m1.cuh"

namespace kvq {

namespace {

// CTAs of W warps per SM, by registers: O takes D / 4 a thread and n-tile
template <int NT, int W> __host__ __device__ constexpr int ctas_per_sm()
{
    const int n = (NT == 1 ? 16 : NT == 2 ? 12 : 8) / W;
    return n > 0 ? n : 1;
}
constexpr int kUnitTiles = 2;                   // 16-token tiles a warp takes at once
constexpr int kUnitPages = 4 * kUnitTiles;
static_assert(kUnitPages == 8, "a unit's 32 tokens have a lane each");

template <int D>
struct KFrag {
    static constexpr int KW = D / 32;   // words of 8 codes per row and lane
    static constexpr int KB = D / 64;   // blocks of 16 channels they span
    uint32_t x[2][KW];
    uint32_t s[KB];                     // a block's scales of the page's four tokens
};

template <int D>
struct VFrag {
    static constexpr int VW = D / 64;   // words of 8 codes per token and lane
    uint32_t x[4][VW];
    uint32_t s;                         // this lane's block's scales of the page's four tokens
};

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&x)[W], const uint8_t *p)
{
    static_assert(W == 1 || W == 2 || W == 4, "4, 8 or 16 bytes");
    if constexpr (W == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        x[0] = u.x;
        x[1] = u.y;
        x[2] = u.z;
        x[3] = u.w;
    } else if constexpr (W == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        x[0] = u.x;
        x[1] = u.y;
    } else {
        x[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// bits 0..3 -> bytes of all ones
__device__ __forceinline__ uint32_t byte_mask(uint32_t bits)
{
    return ((bits * 0x00204081u) & 0x01010101u) * 0xFFu;
}

}  // namespace

// A warp's ring of units in shared memory.  A lane copies the bytes of its own
// fragments (cp.async) and reads them back itself, so neither needs a barrier.
// Fields of a tile, each [32 lanes][bytes]: K row 0, K row 1, K scales, V codes
// of tokens 0..3, V scale.
template <int D, int NT>
struct Ring {
    static constexpr int kK = D / 8, kKS = D / 16, kV = D / 16, kVS = 4;   // bytes per lane
    static constexpr int kOffKS = 2 * 32 * kK, kOffV = kOffKS + 32 * kKS, kOffVS = kOffV + 4 * 32 * kV;
    static constexpr int kTile = kOffVS + 32 * kVS;
    static constexpr int kUnit = kUnitTiles * kTile;
    static constexpr int kUnits = NT <= 2 ? 2 : 3;
    static constexpr int kBytes = kUnits * kUnit;
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int PENDING>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// The queries as mma B fragments: in registers for one n-tile, in shared memory
// (in fragment order, [D / 32][RW * NT][32 lanes] of 16 bytes) for more.
template <int D, int NT, int RW> __host__ __device__ constexpr int q_bytes() { return NT == 1 ? 0 : RW * NT * D * 16; }

template <int D, int NT>
struct Queries {
    uint32_t f[NT == 1 ? D / 32 : 1][4];
    const uint4 *s;   // this lane's entry of (word 0, this warp's first n-tile)
};

// A unit's S^T = K Q^T
template <int D, int NT, int RW>
__device__ __forceinline__ void scores(const KFrag<D> (&f)[kUnitTiles], uint32_t ks_sel, const Queries<D, NT> &q,
                                       float (&sc)[NT][kUnitTiles][4])
{
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < kUnitTiles; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[j][k][e] = 0.f;
#pragma unroll
    for (int w = 0; w < KFrag<D>::KW; ++w) {
        uint32_t lo[kUnitTiles][4], hi[kUnitTiles][4];
#pragma unroll
        for (int k = 0; k < kUnitTiles; ++k) {
            // the block's scale of this lane's two rows, in both halves
            const uint32_t sb = __byte_perm(f[k].s[w / 2], 0u, ks_sel);
            const uint32_t s0 = cvt_lo(sb), s1 = cvt_hi(sb);
            const uint32_t x0 = f[k].x[0][w], x1 = f[k].x[1][w];
            lo[k][0] = hmul2(e2m1_pair<0>(x0), s0);
            lo[k][1] = hmul2(e2m1_pair<0>(x1), s1);
            lo[k][2] = hmul2(e2m1_pair<1>(x0), s0);
            lo[k][3] = hmul2(e2m1_pair<1>(x1), s1);
            hi[k][0] = hmul2(e2m1_pair<2>(x0), s0);
            hi[k][1] = hmul2(e2m1_pair<2>(x1), s1);
            hi[k][2] = hmul2(e2m1_pair<3>(x0), s0);
            hi[k][3] = hmul2(e2m1_pair<3>(x1), s1);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint32_t b[4];
            if constexpr (NT == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = q.f[w][e];
            } else {
                const uint4 v = q.s[(w * RW * NT + j) * 32];
                b[0] = v.x;
                b[1] = v.y;
                b[2] = v.z;
                b[3] = v.w;
            }
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
                mma_16816(sc[j][k], lo[k], b[0], b[1]);
                mma_16816(sc[j][k], hi[k], b[2], b[3]);
            }
        }
    }
}

// One tile's O^T += V^T P^T
template <int D, int NT>
__device__ __forceinline__ void weigh(const VFrag<D> &f, const uint32_t (&pf)[NT][kUnitTiles][2], float (&o)[NT][D / 16][4], int k)
{
    const uint32_t s01 = cvt_lo(f.s), s23 = cvt_hi(f.s);
#pragma unroll
    for (int w = 0; w < VFrag<D>::VW; ++w) {
        // channels 8w + 2y (z0, y0) and 8w + 2y + 1 (z1, y1) of byte y, two tokens a byte
        constexpr uint32_t M = 0x0F0F0F0Fu;
        const uint32_t z0 = (f.x[0][w] & M) | ((f.x[1][w] << 4) & ~M);
        const uint32_t z1 = ((f.x[0][w] >> 4) & M) | (f.x[1][w] & ~M);
        const uint32_t y0 = (f.x[2][w] & M) | ((f.x[3][w] << 4) & ~M);
        const uint32_t y1 = ((f.x[2][w] >> 4) & M) | (f.x[3][w] & ~M);
        const uint32_t af[4][4] = {
            {hmul2(e2m1_pair<0>(z0), s01), hmul2(e2m1_pair<0>(z1), s01), hmul2(e2m1_pair<0>(y0), s23), hmul2(e2m1_pair<0>(y1), s23)},
            {hmul2(e2m1_pair<1>(z0), s01), hmul2(e2m1_pair<1>(z1), s01), hmul2(e2m1_pair<1>(y0), s23), hmul2(e2m1_pair<1>(y1), s23)},
            {hmul2(e2m1_pair<2>(z0), s01), hmul2(e2m1_pair<2>(z1), s01), hmul2(e2m1_pair<2>(y0), s23), hmul2(e2m1_pair<2>(y1), s23)},
            {hmul2(e2m1_pair<3>(z0), s01), hmul2(e2m1_pair<3>(z1), s01), hmul2(e2m1_pair<3>(y0), s23), hmul2(e2m1_pair<3>(y1), s23)}};
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int j = 0; j < NT; ++j) mma_16816(o[j][4 * w + y], af[y], pf[j][k][0], pf[j][k][1]);
    }
}

// Softmax of a unit: scores to P (fp16, as mma B fragments), sums, and the rescale of O.
template <int D, int NT>
__device__ __forceinline__ void softmax_unit(const float (&sc)[NT][kUnitTiles][4], float qk, float (&ref)[NT][2],
                                             float (&l_run)[NT][2], float (&o)[NT][D / 16][4],
                                             uint32_t (&pf)[NT][kUnitTiles][2])
{
    // A row's reference moves only when a score rises more than 2^8 above
    // it (P and its sum stay below 2^8 times their number), so most units
    // need no maximum over the lanes and no rescale: one vote.
    bool above = false;
    float mx[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float m = fmaxf(sc[j][0][c], sc[j][0][c + 2]);
#pragma unroll
            for (int k = 1; k < kUnitTiles; ++k) m = fmax3(m, sc[j][k][c], sc[j][k][c + 2]);
            mx[j][c] = m * qk;
            above |= mx[j][c] > ref[j][c] + 8.f;
        }
    if (__any_sync(kFull, above)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float corr[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float m = mx[j][c];
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
                const bool move = m > ref[j][c] + 8.f;   // the same on the 8 lanes of a row
                corr[c] = !move ? 1.f : ref[j][c] == -INFINITY ? 0.f : fast_exp2(ref[j][c] - m);
                if (move) ref[j][c] = m;
                l_run[j][c] *= corr[c];
            }
#pragma unroll
            for (int pv = 0; pv < D / 16; ++pv) {
                o[j][pv][0] *= corr[0];
                o[j][pv][2] *= corr[0];
                o[j][pv][1] *= corr[1];
                o[j][pv][3] *= corr[1];
            }
        }
    }
    const float2 qk2 = make_float2(qk, qk);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        // a row that has seen nothing yet: every score is -inf, P = 0
        const float2 nref = make_float2(ref[j][0] == -INFINITY ? 0.f : -ref[j][0], ref[j][1] == -INFINITY ? 0.f : -ref[j][1]);
        float2 sum = make_float2(l_run[j][0], l_run[j][1]);
#pragma unroll
        for (int k = 0; k < kUnitTiles; ++k)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 z = ffma2(make_float2(sc[j][k][2 * r], sc[j][k][2 * r + 1]), qk2, nref);
                const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                sum = fadd2(sum, p);
                pf[j][k][r] = movmatrix_trans(pack_half2(p.x, p.y));
            }
        l_run[j][0] = sum.x;
        l_run[j][1] = sum.y;
    }
}

// NT n-tiles of 8 query rows per warp; RW warps share the same tokens and split
// the query rows, the W / RW groups of warps split the tokens.
// LISTS: the call has top-k lists (a sequence of it may have none).  LPT: the
// sequences are taken longest first.  Both are instances of their own because
// their code, unused, cost the others registers (ragged batch 94 -> 85 us).
// MERGE: the splits of one (sequence, kv head) are one thread-block cluster;
// after a cluster barrier its CTAs merge the partials (the combine's function,
// hence its bits) and write the output themselves.
template <int D, int NT, int RW, int W, bool MERGE, bool LISTS, bool LPT>
__global__ void __launch_bounds__(32 * W, ctas_per_sm<NT, W>()) attn_e2m1_kernel(const AttnArgs a)
{
    constexpr int kQWarps = W, kQThreads = 32 * W;
    constexpr int TW = kQWarps / RW;
    constexpr int kRowsPad = RW * NT * 8;
    constexpr int kRowF = D + 4;                     // m, l, two unused, o[D]
    constexpr int PB = e2m1_page_bytes(D), SO = e2m1_scale_off(D);
    constexpr int CPL = D / 4;                       // K channels per lane
    using KF = KFrag<D>;
    using VF = VFrag<D>;
    using R = Ring<D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];

    const int s = blockIdx.x, g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, t = lane & 3;
    const int rw = warp % RW, tw = warp / RW;
    // Without a top-k list, block tables, lengths and the pages of positions
    // below L - q_len may be read before the preceding kernel (the step's
    // append) has finished; everything else waits for it.
    const bool early = !LISTS && a.early_pages;
    if (!early) grid_dependency_wait();
    launch_dependents();
    SeqPick pick = seq_identity(a, blockIdx.z);
    if constexpr (LPT) {
        if (!__syncthreads_and(lpt_classify(a, smem, W * R::kBytes))) pick = lpt_pick(a, blockIdx.z, smem);
    }
    const int b = pick.b;
    const SplitRange sr = split_range(a, s, b, pick.L, LISTS ? pick.topk_len : 0);
    const int L = sr.L, item0 = sr.item0, item1 = sr.item1;
    const bool topk = LISTS && sr.topk;

    // this lane's places inside a page
    const int page_stride = a.num_kv_heads * PB;   // at most 65535 * 288
    const uint8_t *kpool = static_cast<const uint8_t *>(a.k_cache) + (int64_t)g * PB;
    const uint8_t *vpool = static_cast<const uint8_t *>(a.v_cache) + (int64_t)g * PB;
    const int k_code = t * (CPL / 2), k_scale = SO + t * (4 * KF::KB);
    const int v_code = gid * (D / 16), v_scale = SO + 4 * (gid * D / 128);
    const uint32_t ks_sel = (gid & 1) ? 0x3311u : 0x2200u;   // scale bytes (row, row, row + 8, row + 8)

    // --- dense: a unit is 8 pages; lane l (mod 8) holds page l's number (-1: none) ---
    const int step = TW * kUnitPages;
    int u0 = item0 + tw * kUnitPages;
    const unsigned num_pages = (unsigned)min(a.num_pages, (int64_t)0x80000000ll);
    auto raw_page = [&](int u) {
        const int it = u + (lane & (kUnitPages - 1));
        return it < item1 ? __ldg(sr.bt_row + it) : -1;
    };
    auto checked = [&](int phys, int u) {
        if ((unsigned)phys < num_pages) return phys;
        if (u + (lane & (kUnitPages - 1)) < item1 && rw == 0 && lane < kUnitPages) report(a.err_flag, KVQ_DEV_BAD_PAGE);
        return -1;
    };
    uint8_t *ring = smem + warp * R::kBytes;
    const uint32_t ring_s = smem_u32(ring);
    const uint8_t *k_rows = kpool + k_code + (gid & 1) * (D / 2), *k_scales = kpool + k_scale;
    const uint8_t *v_rows = vpool + v_code, *v_scales = vpool + v_scale;
    // Copies of a unit into ring slot `slot`.  Missing pages are read from page 0 and masked.
    auto fetch = [&](int phys, int slot) {
        const int page = max(phys, 0);
#pragma unroll
        for (int k = 0; k < kUnitTiles; ++k) {
            const uint32_t dst = ring_s + slot * R::kUnit + k * R::kTile;
            // (a 32 x 32 -> 64-bit multiply-add each)
            const int kp = __shfl_sync(kFull, page, 4 * k + (gid >> 1)), vp = __shfl_sync(kFull, page, 4 * k + t);
            const uint8_t *kr = k_rows + (int64_t)kp * page_stride, *ks = k_scales + (int64_t)kp * page_stride;
            const uint8_t *vr = v_rows + (int64_t)vp * page_stride, *vs = v_scales + (int64_t)vp * page_stride;
            copy_async<R::kK>(dst + lane * R::kK, kr);
            copy_async<R::kK>(dst + 32 * R::kK + lane * R::kK, kr + D);
            copy_async<R::kKS>(dst + R::kOffKS + lane * R::kKS, ks);
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_async<R::kV>(dst + R::kOffV + j * 32 * R::kV + lane * R::kV, vr + j * (D / 2));
            copy_async<R::kVS>(dst + R::kOffVS + lane * R::kVS, vs);
        }
    };
    int pg[R::kUnits];                     // pages of the units in flight, the next one first
    bool waited = !early;
    if (!topk) {
#pragma unroll
        for (int d = 0; d < R::kUnits; ++d) pg[d] = raw_page(u0 + d * step);
#pragma unroll
        for (int d = 0; d < R::kUnits; ++d) {
            const int u = u0 + d * step;
            if (u < item1) {
                if (!waited && u + kUnitPages > max(L - a.q_len, 0) / 4) {
                    grid_dependency_wait();
                    waited = true;
                }
                pg[d] = checked(pg[d], u);
                fetch(pg[d], d);
            }
            copy_commit();
        }
    }
    if (!waited) grid_dependency_wait();
    if (threadIdx.x == 0) {
        if (!sr.len_ok) report(a.err_flag, KVQ_DEV_BAD_LEN);
        if (LISTS && sr.len_ok && pick.topk_len > a.max_topk) report(a.err_flag, KVQ_DEV_BAD_TOPK);
    }

    float o[NT][D / 16][4];
    float ref[NT][2], l_run[NT][2];       // log2-domain reference of a row, sum of its 2^(s - ref)
    // last position that column c of n-tile j sees (rows that do not exist see everything);
    // needed on masked units only
    auto lim = [&](int j, int c) {
        const int r = (rw * NT + j) * 8 + 2 * t + c;
        return r < a.rows ? L - a.q_len + r / a.group : 0x7FFFFFFE;
    };
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            ref[j][c] = -INFINITY;
            l_run[j][c] = 0.f;
        }
#pragma unroll
        for (int pv = 0; pv < D / 16; ++pv)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][pv][e] = 0.f;
    }
    // query row `row`'s channels t CPL + 8 w .. + 7: the B fragments of the two k-steps of word w
    auto q_words = [&](int row, int w) {
        if (row >= a.rows) return make_uint4(0u, 0u, 0u, 0u);
        const int i = row / a.group, h = g * a.group + row % a.group;
        return *reinterpret_cast<const uint4 *>(static_cast<const __half *>(a.q) +
                                                (((int64_t)b * a.q_len + i) * a.num_q_heads + h) * D + t * CPL + 8 * w);
    };
    Queries<D, NT> qs;
    if constexpr (NT == 1) {
#pragma unroll
        for (int w = 0; w < KF::KW; ++w) {
            const uint4 v = q_words(gid, w);
            qs.f[w][0] = v.x;
            qs.f[w][1] = v.y;
            qs.f[w][2] = v.z;
            qs.f[w][3] = v.w;
        }
    } else {
        uint4 *qm = reinterpret_cast<uint4 *>(smem + kQWarps * R::kBytes);
        for (int i = warp; i < KF::KW * RW * NT; i += kQWarps)
            qm[i * 32 + lane] = q_words((i % (RW * NT)) * 8 + gid, i / (RW * NT));
        __syncthreads();
        qs.s = qm + rw * NT * 32 + lane;
    }
    const float qk = a.qk_scale_log2;
    float sc[NT][kUnitTiles][4];
    uint32_t pf[NT][kUnitTiles][2];
    constexpr int kNoToken = 0x7FFFFFFF;   // a position beyond every row's limit

    if (!topk) {
        const int clean_end = (L - a.q_len + 1) / 4;     // pages below hold only positions that every row sees
        int next = raw_page(u0 + R::kUnits * step);
        for (int slot = 0; u0 < item1; u0 += step) {
            const int u = u0 + R::kUnits * step;         // the unit this slot holds next
            const int ahead = raw_page(u + step);        // (the block table is read a unit before it is used)
            copy_wait<R::kUnits - 1>();
            const uint8_t *un = ring + slot * R::kUnit;
            {
                KF f[kUnitTiles];
#pragma unroll
                for (int k = 0; k < kUnitTiles; ++k) {
                    const uint8_t *tl = un + k * R::kTile;
                    load_words(f[k].x[0], tl + lane * R::kK);
                    load_words(f[k].x[1], tl + 32 * R::kK + lane * R::kK);
                    load_words(f[k].s, tl + R::kOffKS + lane * R::kKS);
                }
                scores<D, NT, RW>(f, ks_sel, qs, sc);
            }
            uint32_t vmask[kUnitTiles];
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) vmask[k] = 0xFFFFFFFFu;
            const unsigned paged = __ballot_sync(kFull, pg[0] >= 0);   // bits 0..7 (and their copies): pages
            if (paged != kFull || u0 + kUnitPages > clean_end) {
                // Slots without a token may hold any bits: their scores are replaced (whatever they
                // are), and their V scales zeroed, since a NaN scale times a probability of 0 is NaN.
                const unsigned live = __ballot_sync(kFull, ((paged >> (lane >> 2)) & 1u) && u0 * 4 + lane < L);
#pragma unroll
                for (int k = 0; k < kUnitTiles; ++k) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int e = 16 * k + 4 * (gid >> 1) + (gid & 1) + 2 * r;
                        const int pos = ((live >> e) & 1u) ? u0 * 4 + e : kNoToken;
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (pos > lim(j, c)) sc[j][k][2 * r + c] = -INFINITY;
                    }
                    vmask[k] = byte_mask((live >> (16 * k + 4 * t)) & 15u);
                }
            }
            softmax_unit<D, NT>(sc, qk, ref, l_run, o, pf);
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
                const uint8_t *tl = un + k * R::kTile;
                VF f;
#pragma unroll
                for (int j = 0; j < 4; ++j) load_words(f.x[j], tl + R::kOffV + j * 32 * R::kV + lane * R::kV);
                f.s = *reinterpret_cast<const uint32_t *>(tl + R::kOffVS + lane * R::kVS) & vmask[k];
                weigh<D, NT>(f, pf, o, k);
            }
            // this slot has been read (by this lane alone)
#pragma unroll
            for (int d = 0; d + 1 < R::kUnits; ++d) pg[d] = pg[d + 1];
            pg[R::kUnits - 1] = checked(next, u);
            next = ahead;
            if (u < item1) fetch(pg[R::kUnits - 1], slot);
            copy_commit();
            slot = slot + 1 == R::kUnits ? 0 : slot + 1;
        }
    }
    if constexpr (LISTS) if (topk) {
        // --- top-k: a unit is 32 list entries; entry 16 k + 4 p + j is token j of page slot p of
        // tile k; lane l holds entry l's position (-1: none) and page ---
        const int32_t *list = a.topk_idx + ((int64_t)b * a.num_kv_heads + g) * a.max_topk;
        for (int e0 = item0 + tw * 32; e0 < item1; e0 += TW * 32) {
            int pos = e0 + lane < item1 ? __ldg(list + e0 + lane) : -1;
            int phys = 0;
            if (e0 + lane < item1 && (pos < 0 || pos >= L)) {
                if (rw == 0) report(a.err_flag, KVQ_DEV_BAD_TOPK);
                pos = -1;
            }
            if (pos >= 0) {
                phys = __ldg(sr.bt_row + (pos >> 2));
                if (phys < 0 || (int64_t)phys >= a.num_pages) {
                    if (rw == 0) report(a.err_flag, KVQ_DEV_BAD_PAGE);
                    pos = -1;
                    phys = 0;
                }
            }
            const unsigned live = __ballot_sync(kFull, pos >= 0);
            KF kf[kUnitTiles];
            int row_pos[kUnitTiles][2];
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
                KF &f = kf[k];
#pragma unroll
                for (int w = 0; w < KF::KB; ++w) f.s[w] = 0u;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int e = 16 * k + 4 * (gid >> 1) + (gid & 1) + 2 * r;
                    const int p = __shfl_sync(kFull, pos, e), at = p & 3;
                    const uint8_t *row = kpool + (int64_t)__shfl_sync(kFull, phys, e) * page_stride;
                    row_pos[k][r] = p >= 0 ? p : kNoToken;
                    load_words(f.x[r], row + k_code + at * (D / 2));
#pragma unroll
                    for (int w = 0; w < KF::KB; ++w) f.s[w] |= (uint32_t)row[k_scale + 4 * w + at] << (8 * ((gid & 1) + 2 * r));
                }
            }
            scores<D, NT, RW>(kf, ks_sel, qs, sc);
            VF vf[kUnitTiles];
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
                vf[k].s = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int e = 16 * k + 4 * t + j;
                    const int at = __shfl_sync(kFull, pos, e) & 3;
                    const uint8_t *row = vpool + (int64_t)__shfl_sync(kFull, phys, e) * page_stride;
                    load_words(vf[k].x[j], row + v_code + at * (D / 2));
                    vf[k].s |= (uint32_t)row[v_scale + at] << (8 * j);
                }
                vf[k].s &= byte_mask((live >> (16 * k + 4 * t)) & 15u);
            }
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (row_pos[k][e >> 1] > lim(j, e & 1)) sc[j][k][e] = -INFINITY;
            softmax_unit<D, NT>(sc, qk, ref, l_run, o, pf);
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) weigh<D, NT>(vf[k], pf, o, k);
        }
    }
    copy_wait<0>();     // the last groups are empty
    __syncthreads();    // the merge reuses the rings

    // ---- the warps' results to shared memory, merged, to the workspace ----
    float *mbuf = reinterpret_cast<float *>(smem);       // [TW][kRowsPad][kRowF]
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float l = l_run[j][c];
            l += __shfl_xor_sync(kFull, l, 4);
            l += __shfl_xor_sync(kFull, l, 8);
            l += __shfl_xor_sync(kFull, l, 16);
            float *dst = mbuf + (tw * kRowsPad + (rw * NT + j) * 8 + 2 * t + c) * kRowF;
            if (gid == 0) {
                dst[0] = ref[j][c];
                dst[1] = l;
            }
            // lane (gid, t): the D / 8 channels from gid D / 8 on, a pair per P V tile
#pragma unroll
            for (int pv = 0; pv < D / 16; ++pv)
                *reinterpret_cast<float2 *>(dst + 4 + gid * (D / 8) + 2 * pv) = make_float2(o[j][pv][c], o[j][pv][c + 2]);
        }
    __syncthreads();
    const int S = a.num_splits;
    for (int idx = threadIdx.x * 4; idx < a.rows * D; idx += kQThreads * 4) {
        const int row = idx / D, d = idx % D;
        float M = -INFINITY;
#pragma unroll
        for (int q = 0; q < TW; ++q) M = fmaxf(M, mbuf[(q * kRowsPad + row) * kRowF]);
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < TW; ++q) {
            const float *src = mbuf + (q * kRowsPad + row) * kRowF;
            const float w = M == -INFINITY ? 0.f : fast_exp2(src[0] - M);
            lsum += w * src[1];
            const float4 x = *reinterpret_cast<const float4 *>(src + 4 + d);
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        }
        const int i = row / a.group, h = g * a.group + row % a.group;
        const int64_t unit = (((int64_t)b * a.num_q_heads + h) * a.q_len + i) * S + s;
        // A NaN score makes the row NaN: the split then outweighs every other in the combine, which
        // leaves a split out by l alone.
        const bool nan = lsum != lsum;
        if (d == 0) {
            a.ws_m[unit] = nan ? FLT_MAX : lsum > 0.f ? M * kLn2 : -INFINITY;
            a.ws_l[unit] = nan ? 1.f : lsum;
        }
        if (lsum == 0.f) continue;                        // an empty row: its partial stays unwritten
        const float inv = a.out_scale / lsum;
        *reinterpret_cast<float4 *>(a.ws_o + unit * D + d) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    if constexpr (MERGE) {
        cluster_barrier();   // release, then acquire: the cluster's workspace stores are visible
        for (int row = s + S * warp; row < a.rows; row += S * kQWarps) {
            const int i = row / a.group, h = g * a.group + row % a.group;
            const int64_t r = ((int64_t)b * a.num_q_heads + h) * a.q_len + i;
            float acc[D / 32];
            const float sum = merge_splits<D>(a.ws_o + r * S * D, a.ws_m + r * S, a.ws_l + r * S, S, lane, 0, 1, acc);
            store_merged<D>(static_cast<__half *>(a.out), b, i, h, a.q_len, a.num_q_heads, lane, acc, sum);
        }
    }
}

// ---------------------------------------------------------------------------

template <int D, int NT, int RW, int W, bool MERGE, bool LISTS, bool LPT = false>
static cudaError_t launch_e2m1(const AttnArgs &a, cudaStream_t stream)
{
    constexpr int merge = W * NT * 8 * (D + 4) * 4, ring = W * Ring<D, NT>::kBytes + q_bytes<D, NT, RW>();
    constexpr int bytes = merge > ring ? merge : ring;
    static_assert(bytes <= 232448, "shared memory exceeds one CTA's limit");
    static uint64_t configured = 0;   // one bit per device ordinal
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
        e = cudaFuncSetAttribute(attn_e2m1_kernel<D, NT, RW, W, MERGE, LISTS, LPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_splits, a.num_kv_heads, a.batch);
    cfg.blockDim = dim3(32 * W);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.num_splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = MERGE ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, attn_e2m1_kernel<D, NT, RW, W, MERGE, LISTS, LPT>, a);
}

// The CTAs of W = 4 warps that are resident at once.
static inline int64_t e2m1_resident(int rows)
{
    const int tiles = (rows + 7) / 8;
    return int64_t(device_sm_count()) *
           (tiles <= 1 ? ctas_per_sm<1, 4>() : tiles <= 2 ? ctas_per_sm<2, 4>() : ctas_per_sm<4, 4>());
}

// A grid that leaves most of the card idle takes wider CTAs: the same splits, each
// walked by two or four times as many warps.
template <int D, int NT, int RW, bool MERGE, bool LISTS>
static cudaError_t launch_e2m1_width(const AttnArgs &a, cudaStream_t stream)
{
    const int64_t ctas = int64_t(a.batch) * a.num_kv_heads * a.num_splits, resident = e2m1_resident(a.rows);
    // (a cluster's CTAs share a GPC: one of more than four CTAs that each fill an SM may not find room)
    const int units = (a.max_pages / a.num_splits + kUnitPages - 1) / kUnitPages;   // of a full split
    if constexpr (NT == 1)
        if (units > 8 && (MERGE ? a.num_splits <= 4 && ctas <= 128 : ctas * 4 <= resident))
            return launch_e2m1<D, NT, RW, 16, MERGE, LISTS>(a, stream);
    if (units > 4 && ctas * 2 <= resident) return launch_e2m1<D, NT, RW, 8, MERGE, LISTS>(a, stream);
    if constexpr (!MERGE)   // (MERGE: one wave)
        if (a.longest_first) return launch_e2m1<D, NT, RW, 4, MERGE, LISTS, true>(a, stream);
    return launch_e2m1<D, NT, RW, 4, MERGE, LISTS>(a, stream);
}

template <int D, bool MERGE, bool LISTS>
static cudaError_t launch_e2m1_rows(const AttnArgs &a, cudaStream_t stream)
{
    const int tiles = (a.rows + 7) / 8;
    if (tiles <= 1) return launch_e2m1_width<D, 1, 1, MERGE, LISTS>(a, stream);
    if (tiles <= 2) return launch_e2m1_width<D, 2, 1, MERGE, LISTS>(a, stream);
    if (tiles <= 3) return launch_e2m1_width<D, 3, 1, MERGE, LISTS>(a, stream);
    if (tiles <= 4) return launch_e2m1_width<D, 4, 1, MERGE, LISTS>(a, stream);
    return launch_e2m1_width<D, 4, 2, MERGE, LISTS>(a, stream);
}

template <int D>
static cudaError_t launch_e2m1_dim(const AttnArgs &a, bool merge, cudaStream_t stream)
{
    if (merge) return launch_e2m1_rows<D, true, false>(a, stream);
    return a.topk_idx ? launch_e2m1_rows<D, false, true>(a, stream) : launch_e2m1_rows<D, false, false>(a, stream);
}

}  // namespace kvq
