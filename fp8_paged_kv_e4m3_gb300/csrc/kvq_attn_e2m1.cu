// kvq_attn_e2m1.cu -- split-K paged decode / verify attention over the 4-bit
// (E2M1) cache.
//
// The attention is the split kernel's: s_j = sm_scale k_scale sum_d q_d K_jd,
// out = v_scale sum_j p_j V_j / sum_j p_j with K, V = E2M1(code) * b, an exact
// fp16 value (at most 6 significant bits, magnitude at most 2688), so both
// products run on fp16 tensor-core instructions (mma.sync m16n8k16, tokens on
// M, query rows on N) with binary32 sums and the layer scales hoisted.
//
// One CTA of 4 warps per (split, kv head, sequence); a warp takes units of 32
// tokens (two tiles of four pages) and keeps its own softmax.  A thread loads
// from global memory exactly the bytes of its own matrix fragments, so nothing
// goes through shared memory and no warp waits for another until the merge:
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
#include <cfloat>

#include "kvq_attn_kernel.cuh"
#include "kvq_e2m1.cuh"

namespace kvq {

namespace {

constexpr int kQWarps = 4;
constexpr int kQThreads = 32 * kQWarps;
constexpr int kUnitTiles = 2;                   // 16-token tiles a warp takes at once
constexpr int kUnitPages = 4 * kUnitTiles;

template <int D>
struct Frag {
    static constexpr int KW = D / 32;   // words of 8 codes per K row and lane
    static constexpr int KB = D / 64;   // blocks of 16 channels they span (scale words)
    static constexpr int VW = D / 64;   // words of 8 codes per V token and lane
    uint32_t k[2][KW];
    uint32_t ks[KB];                    // a block's scales of the page's four tokens
    uint32_t v[4][VW];
    uint32_t vs;                        // this lane's block's scales of the page's four tokens
};

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&x)[W], const uint8_t *p)
{
    static_assert(W == 1 || W == 2 || W == 4, "4, 8 or 16 bytes");
    if (W == 4) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        x[0] = u.x;
        x[W > 1 ? 1 : 0] = u.y;
        x[W > 2 ? 2 : 0] = u.z;
        x[W > 3 ? 3 : 0] = u.w;
    } else if (W == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
        x[0] = u.x;
        x[W > 1 ? 1 : 0] = u.y;
    } else {
        x[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
}

template <int W>
__device__ __forceinline__ void zero_words(uint32_t (&x)[W])
{
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = 0u;
}

}  // namespace

// NT n-tiles of 8 query rows per warp; RW warps share the same tokens and split
// the query rows, the 4 / RW groups of warps split the tokens.
template <int D, int NT, int RW>
__global__ void __launch_bounds__(kQThreads, NT == 1 ? 4 : 3) attn_e2m1_kernel(const AttnArgs a)
{
    constexpr int TW = kQWarps / RW;
    constexpr int kRowsPad = RW * NT * 8;
    constexpr int kRowF = D + 4;                     // m, l, two unused, o[D]
    constexpr int PB = e2m1_page_bytes(D), SO = e2m1_scale_off(D);
    constexpr int CPL = D / 4;                       // K channels per lane
    using F = Frag<D>;
    extern __shared__ __align__(16) uint8_t smem[];

    const int s = blockIdx.x, g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, t = lane & 3;
    const int rw = warp % RW, tw = warp / RW;
    grid_dependency_wait();
    launch_dependents();
    const SeqPick pick = seq_identity(a, blockIdx.z);
    const int b = pick.b;
    const SplitRange sr = split_range(a, s, b, pick.L, pick.topk_len);
    const int L = sr.L, item0 = sr.item0, item1 = sr.item1;
    const bool topk = sr.topk;
    if (threadIdx.x == 0) {
        if (!sr.len_ok) report(a.err_flag, KVQ_DEV_BAD_LEN);
        if (sr.len_ok && pick.topk_len > a.max_topk) report(a.err_flag, KVQ_DEV_BAD_TOPK);
    }

    float o[NT][D / 16][4];
    float m_run[NT][2], l_run[NT][2];
    uint32_t qf[NT][D / 16][2];
    int lim[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int row = (rw * NT + j) * 8 + gid;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = (rw * NT + j) * 8 + 2 * t + c;
            lim[j][c] = (r < a.rows) ? L - a.q_len + r / a.group : 0x7FFFFFFF;
            m_run[j][c] = -INFINITY;
            l_run[j][c] = 0.f;
        }
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            qf[j][ks][0] = qf[j][ks][1] = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][ks][e] = 0.f;
        }
        if (row < a.rows) {
            const int i = row / a.group, h = g * a.group + row % a.group;
            const __half *qrow = static_cast<const __half *>(a.q) +
                                 (((int64_t)b * a.q_len + i) * a.num_q_heads + h) * D + t * CPL;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint2 v = *reinterpret_cast<const uint2 *>(qrow + 4 * ks);
                qf[j][ks][0] = v.x;
                qf[j][ks][1] = v.y;
            }
        }
    }
    const uint8_t *kpool = static_cast<const uint8_t *>(a.k_cache);
    const uint8_t *vpool = static_cast<const uint8_t *>(a.v_cache);
    const int first_masked = L - a.q_len + 1;        // positions from here on are masked for some row
    const uint32_t ks_sel = (gid & 1) ? 0x3311u : 0x2200u;   // scale bytes (row, row, row + 8, row + 8)

    const int ipu = topk ? 4 * kUnitPages : kUnitPages;   // items per unit: pages or list entries
    const int32_t *list = topk ? a.topk_idx + ((int64_t)b * a.num_kv_heads + g) * a.max_topk : nullptr;
    for (int u0 = item0 + tw * ipu; u0 < item1; u0 += TW * ipu) {
        F f[kUnitTiles];
        int kpos[kUnitTiles][2];          // positions of this lane's K rows, -1 = no token
        uint32_t vlive[kUnitTiles];       // 0xFF in byte j: token j of this lane's V page holds a token
        bool need_mask;
        if (!topk) {
            const int it = u0 + (lane & (kUnitPages - 1));
            int phys = it < item1 ? __ldg(sr.bt_row + it) : -1;
            const bool bad = it < item1 && (phys < 0 || (int64_t)phys >= a.num_pages);
            if (bad) phys = -1;
            if (bad && rw == 0 && lane < kUnitPages) report(a.err_flag, KVQ_DEV_BAD_PAGE);
            need_mask = __any_sync(kFull, phys < 0) || (u0 + kUnitPages) * 4 > first_masked;
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
                const int kp = __shfl_sync(kFull, phys, 4 * k + (gid >> 1));
                const int vp = __shfl_sync(kFull, phys, 4 * k + t);
                const int kpos0 = (u0 + 4 * k + (gid >> 1)) * 4 + (gid & 1);
                kpos[k][0] = kp >= 0 ? kpos0 : -1;
                kpos[k][1] = kp >= 0 ? kpos0 + 2 : -1;
                const int vleft = vp >= 0 ? L - (u0 + 4 * k + t) * 4 : 0;   // tokens of the page inside the context
                vlive[k] = vleft >= 4 ? 0xFFFFFFFFu : vleft <= 0 ? 0u : (1u << (8 * vleft)) - 1u;
                zero_words(f[k].k[0]);
                zero_words(f[k].k[1]);
                zero_words(f[k].ks);
                if (kp >= 0) {
                    const uint8_t *pg = kpool + ((int64_t)kp * a.num_kv_heads + g) * PB;
                    load_words(f[k].k[0], pg + (gid & 1) * (D / 2) + t * (CPL / 2));
                    load_words(f[k].k[1], pg + (2 + (gid & 1)) * (D / 2) + t * (CPL / 2));
                    load_words(f[k].ks, pg + SO + t * (4 * F::KB));
                }
                f[k].vs = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) zero_words(f[k].v[j]);
                if (vp >= 0) {
                    const uint8_t *pg = vpool + ((int64_t)vp * a.num_kv_heads + g) * PB;
#pragma unroll
                    for (int j = 0; j < 4; ++j) load_words(f[k].v[j], pg + j * (D / 2) + gid * (D / 16));
                    f[k].vs = __ldg(reinterpret_cast<const uint32_t *>(pg + SO + 4 * (gid * D / 128)));
                }
            }
        } else {
            // entry 16 k + 4 p + j of the unit is token j of page slot p of tile k
            const int it = u0 + lane;
            const bool exists = it < item1;
            int idx = exists ? __ldg(list + it) : -1;
            const bool idx_ok = idx >= 0 && idx < L;
            if (exists && !idx_ok && rw == 0) report(a.err_flag, KVQ_DEV_BAD_TOPK);
            int phys = idx_ok ? __ldg(sr.bt_row + (idx >> 2)) : -1;
            if (idx_ok && (phys < 0 || (int64_t)phys >= a.num_pages)) {
                if (rw == 0) report(a.err_flag, KVQ_DEV_BAD_PAGE);
                phys = -1;
            }
            if (phys < 0) idx = -1;
            need_mask = true;
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
                zero_words(f[k].ks);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int e = 16 * k + 4 * (gid >> 1) + (gid & 1) + 2 * r;
                    const int kp = __shfl_sync(kFull, phys, e), ki = __shfl_sync(kFull, idx, e);
                    kpos[k][r] = ki;
                    zero_words(f[k].k[r]);
                    if (ki >= 0) {
                        const uint8_t *pg = kpool + ((int64_t)kp * a.num_kv_heads + g) * PB;
                        load_words(f[k].k[r], pg + (ki & 3) * (D / 2) + t * (CPL / 2));
#pragma unroll
                        for (int w = 0; w < F::KB; ++w)
                            f[k].ks[w] |= (uint32_t)__ldg(pg + SO + 4 * (t * F::KB + w) + (ki & 3))
                                          << (8 * ((gid & 1) + 2 * r));
                    }
                }
                f[k].vs = 0u;
                vlive[k] = 0xFFFFFFFFu;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int e = 16 * k + 4 * t + j;
                    const int vp = __shfl_sync(kFull, phys, e), vi = __shfl_sync(kFull, idx, e);
                    zero_words(f[k].v[j]);
                    if (vi >= 0) {
                        const uint8_t *pg = vpool + ((int64_t)vp * a.num_kv_heads + g) * PB;
                        load_words(f[k].v[j], pg + (vi & 3) * (D / 2) + gid * (D / 16));
                        f[k].vs |= (uint32_t)__ldg(pg + SO + 4 * (gid * D / 128) + (vi & 3)) << (8 * j);
                    }
                }
            }
        }

        // ---- S^T = K Q^T ----
        float sc[NT][kUnitTiles][4];
#pragma unroll
        for (int k = 0; k < kUnitTiles; ++k) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][k][e] = 0.f;
#pragma unroll
            for (int w = 0; w < F::KW; ++w) {
                // the block's scale of this lane's two rows, in both halves
                const uint32_t sb = __byte_perm(f[k].ks[w / 2], 0u, ks_sel);
                const uint32_t s0 = cvt_lo(sb), s1 = cvt_hi(sb);
                const uint32_t x0 = f[k].k[0][w], x1 = f[k].k[1][w];
                const uint32_t lo[4] = {hmul2(e2m1_pair<0>(x0), s0), hmul2(e2m1_pair<0>(x1), s1),
                                        hmul2(e2m1_pair<1>(x0), s0), hmul2(e2m1_pair<1>(x1), s1)};
                const uint32_t hi[4] = {hmul2(e2m1_pair<2>(x0), s0), hmul2(e2m1_pair<2>(x1), s1),
                                        hmul2(e2m1_pair<3>(x0), s0), hmul2(e2m1_pair<3>(x1), s1)};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma_16816(sc[j][k], lo, qf[j][2 * w][0], qf[j][2 * w][1]);
                    mma_16816(sc[j][k], hi, qf[j][2 * w + 1][0], qf[j][2 * w + 1][1]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][k][e] *= a.qk_scale_log2;
        }
        if (need_mask) {
            // Slots without a token may hold any bits: their scores are replaced (whatever they
            // are), and their V scales zeroed, since a NaN scale times a probability of 0 is NaN.
#pragma unroll
            for (int k = 0; k < kUnitTiles; ++k) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int pos = kpos[k][e >> 1];
                        if (!(pos >= 0 && pos <= lim[j][e & 1])) sc[j][k][e] = -INFINITY;
                    }
                f[k].vs &= vlive[k];
            }
        }
        // ---- online softmax (a column's rows lie on the 8 lanes that share t) ----
        float corr[NT][2];
        bool raised = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = fmaxf(sc[j][0][c], sc[j][0][c + 2]);
#pragma unroll
                for (int k = 1; k < kUnitTiles; ++k) mx = fmaxf(mx, fmaxf(sc[j][k][c], sc[j][k][c + 2]));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                const float m_new = fmaxf(m_run[j][c], mx);
                const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
                const bool up = m_new != m_run[j][c];
                corr[j][c] = up ? fast_exp2(m_run[j][c] - m_use) : 1.f;
                raised |= up;
                m_run[j][c] = m_new;
                float lsum = l_run[j][c] * corr[j][c];
#pragma unroll
                for (int k = 0; k < kUnitTiles; ++k) {
                    sc[j][k][c] = fast_exp2(sc[j][k][c] - m_use);
                    sc[j][k][c + 2] = fast_exp2(sc[j][k][c + 2] - m_use);
                    lsum += sc[j][k][c] + sc[j][k][c + 2];
                }
                l_run[j][c] = lsum;
            }
        if (__any_sync(kFull, raised)) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int pv = 0; pv < D / 16; ++pv) {
                    o[j][pv][0] *= corr[j][0];
                    o[j][pv][2] *= corr[j][0];
                    o[j][pv][1] *= corr[j][1];
                    o[j][pv][3] *= corr[j][1];
                }
        }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int k = 0; k < kUnitTiles; ++k) {
            uint32_t pf[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                pf[j][0] = movmatrix_trans(pack_half2(sc[j][k][0], sc[j][k][1]));
                pf[j][1] = movmatrix_trans(pack_half2(sc[j][k][2], sc[j][k][3]));
            }
            const uint32_t s01 = cvt_lo(f[k].vs), s23 = cvt_hi(f[k].vs);
#pragma unroll
            for (int w = 0; w < F::VW; ++w) {
                // channels 8w + 2y (z0) and 8w + 2y + 1 (z1) of byte y, two tokens a byte
                constexpr uint32_t M = 0x0F0F0F0Fu;
                const uint32_t z0 = (f[k].v[0][w] & M) | ((f[k].v[1][w] << 4) & ~M);
                const uint32_t z1 = ((f[k].v[0][w] >> 4) & M) | (f[k].v[1][w] & ~M);
                const uint32_t y0 = (f[k].v[2][w] & M) | ((f[k].v[3][w] << 4) & ~M);
                const uint32_t y1 = ((f[k].v[2][w] >> 4) & M) | (f[k].v[3][w] & ~M);
                const uint32_t af[4][4] = {
                    {hmul2(e2m1_pair<0>(z0), s01), hmul2(e2m1_pair<0>(z1), s01), hmul2(e2m1_pair<0>(y0), s23), hmul2(e2m1_pair<0>(y1), s23)},
                    {hmul2(e2m1_pair<1>(z0), s01), hmul2(e2m1_pair<1>(z1), s01), hmul2(e2m1_pair<1>(y0), s23), hmul2(e2m1_pair<1>(y1), s23)},
                    {hmul2(e2m1_pair<2>(z0), s01), hmul2(e2m1_pair<2>(z1), s01), hmul2(e2m1_pair<2>(y0), s23), hmul2(e2m1_pair<2>(y1), s23)},
                    {hmul2(e2m1_pair<3>(z0), s01), hmul2(e2m1_pair<3>(z1), s01), hmul2(e2m1_pair<3>(y0), s23), hmul2(e2m1_pair<3>(y1), s23)}};
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma_16816(o[j][4 * w + y], af[y], pf[j][0], pf[j][1]);
            }
        }
    }

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
                dst[0] = m_run[j][c];
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
}

// ---------------------------------------------------------------------------

template <int D, int NT, int RW>
static cudaError_t launch_e2m1(const AttnArgs &a, cudaStream_t stream)
{
    constexpr int bytes = (kQWarps / RW) * RW * NT * 8 * (D + 4) * 4;
    static uint64_t configured = 0;   // one bit per device ordinal
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
        e = cudaFuncSetAttribute(attn_e2m1_kernel<D, NT, RW>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    return launch_pdl(attn_e2m1_kernel<D, NT, RW>, dim3(a.num_splits, a.num_kv_heads, a.batch), dim3(kQThreads), bytes,
                      stream, a);
}

template <int D>
static cudaError_t launch_e2m1_rows(const AttnArgs &a, cudaStream_t stream)
{
    const int tiles = (a.rows + 7) / 8;
    if (tiles <= 1) return launch_e2m1<D, 1, 1>(a, stream);
    if (tiles <= 2) return launch_e2m1<D, 2, 1>(a, stream);
    if (tiles <= 4) return launch_e2m1<D, 2, 2>(a, stream);
    return launch_e2m1<D, 2, 4>(a, stream);
}

cudaError_t launch_attention_e2m1(int head_dim, const AttnArgs &a, cudaStream_t stream)
{
    if (a.batch == 0) return cudaSuccess;
    return head_dim == 128 ? launch_e2m1_rows<128>(a, stream) : launch_e2m1_rows<64>(a, stream);
}

}  // namespace kvq
