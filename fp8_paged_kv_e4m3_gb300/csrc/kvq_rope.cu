// kvq_rope.cu -- rotary positions applied on the way into the paged cache,
// the plain append to the E2M1 cache, and the E2M1 cache's read-back.
//
// Rotation of the channel pair (x1, x2) of a token at position p, with
// c = cos and s = sin of its angle p * f_j (times the table's factor):
//     y1 = fl(fl(x1 c) - fl(x2 s)),   y2 = fl(fl(x2 c) + fl(x1 s))
// in binary32.  The queries are rounded to fp16 once; the keys go from these
// binary32 values straight to the pool's type, one rounding (through fp16
// first, a key would be rounded twice).
//
// Bound by memory: every element is read once and written once.  8192 tokens,
// 32 query and 4 kv heads of 128 channels: into E4M3 pages 30.0 us (80 % of the
// copy peak over the 164 MB moved); 8240 tokens into E2M1 pages, half of the
// channels rotated, and their rows read back 35.5 us (75 %), where the maximum,
// the quotient and the reciprocal of each block of 16 channels keep the ALU 41 %
// busy; 4096 tokens of 8 kv heads appended to E2M1 pages without a rotation and
// read back 12.7 us (43 MB).  The few tokens of a decode step take 2.3 to 4.0 us,
// a launch and two dependent reads.
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_e2m1.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRopeThreads = 256;

// eight fp16 <-> eight fp32
__device__ __forceinline__ void unpack8(uint4 h, float (&x)[8])
{
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8])
{
    return make_uint4(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]), pack_half2(y[4], y[5]), pack_half2(y[6], y[7]));
}

// eight fp32 -> eight E4M3 bytes, each divided by the scale in binary32
__device__ __forceinline__ uint2 quantize8(const float (&y)[8], float scale)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[2 * i], scale), __fdiv_rn(y[2 * i + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

}  // namespace

// ---------------------------------------------------------------------------
// Append with the rotation on the way.  A lane owns 8 consecutive channels of a
// head, a warp holds whole heads (D / 8 lanes each), so that a pair's other half
// comes from a lane of the warp (half layout: half / 8 lanes away; interleaved:
// the lane itself) and rotating the queries in place is safe: every load precedes
// the shuffles, every store follows them.  A warp takes one token and, by
// blockIdx.y, some of its query heads or of its key and value heads, kIter groups
// of heads at a time: all of a group's loads first, the table entries (which every
// head of the token shares) once.  D = 0: any head_dim.
constexpr int kIter = 4;

// max |x| over eight values, as binary32 bits; NaN if any is (maximum of three, sm_100 and later)
__device__ __forceinline__ uint32_t absmax8_bits(const float (&x)[8])
{
    float a, b, c;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(x[3]), "f"(x[4]), "f"(x[5]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(c) : "f"(x[6]), "f"(x[7]), "f"(a));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(b), "f"(c));
    return __float_as_uint(a);
}

// c, s: this lane's table entries, s with the sign of its half: out = fl(x c) + fl(partner s).
// (As packed two-lane multiplies and adds this is compiled to fused multiply-adds, which
// round once: the scalar intrinsics keep the three roundings of the definition.)
__device__ __forceinline__ void rotate8(float (&x)[8], uint4 other, bool interleaved, const float (&c)[8], const float (&s)[8])
{
    float p[8];
    unpack8(other, p);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(interleaved ? p[j ^ 1] : p[j], s[j]));
}

// This lane's table entries for position `pos`: c, and s with the sign of the lane's half.
__device__ __forceinline__ void load_turn(const RopeArgs &a, int pos, int ch, float (&c)[8], float (&s)[8])
{
    const int half = a.rot_dim / 2;
    const float *row = a.table + (int64_t)pos * a.rot_dim;
    if (a.interleaved) {
        const float4 cc = __ldg(reinterpret_cast<const float4 *>(row + ch / 2));
        const float4 ss = __ldg(reinterpret_cast<const float4 *>(row + half + ch / 2));
        const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = cv[j / 2];
            s[j] = (j & 1) ? sv[j / 2] : -sv[j / 2];
        }
    } else {
        const bool lower = ch < half;
        const int at = lower ? ch : ch - half;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 cc = __ldg(reinterpret_cast<const float4 *>(row + at) + q);
            const float4 ss = __ldg(reinterpret_cast<const float4 *>(row + half + at) + q);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[4 * q + j] = cv[j];
                s[4 * q + j] = lower ? -sv[j] : sv[j];
            }
        }
    }
}

__device__ __forceinline__ uint4 shuffle4(uint4 v, int lane)
{
    return make_uint4(__shfl_sync(kAll, v.x, lane), __shfl_sync(kAll, v.y, lane), __shfl_sync(kAll, v.z, lane),
                      __shfl_sync(kAll, v.w, lane));
}

template <PoolKind POOL, bool ROTATE, int D>
__global__ void __launch_bounds__(kRopeThreads, 4) append_rope_kernel(const RopeArgs a)
{
    grid_dependency_wait();   // the projections and indices may come from the previous kernel
    launch_dependents();
    const int head_dim = D ? D : a.head_dim;
    const int lanes = head_dim / 8, hpw = 32 / lanes;   // lanes per head, heads per warp
    const int lane = threadIdx.x & 31;
    const int64_t token = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (token >= a.num_tokens) return;
    const int sub = lane / lanes, vec = lane - sub * lanes;   // the warp's head this lane belongs to, its vector
    const int ch = vec * 8;
    const bool live = sub < hpw;                        // lanes past the last whole head idle
    const int within = sub * head_dim + ch;             // this lane's place in a group of hpw heads
    const int group_dim = hpw * head_dim;
    const int pos = ROTATE ? __ldg(a.positions + token) : 0;
    const bool pos_ok = !ROTATE || (unsigned)pos < (unsigned)a.max_positions;
    const bool turns = ROTATE && ch < a.rot_dim;
    const int half = a.rot_dim / 2;
    const int mate = a.interleaved || !turns ? lane : (ch < half ? lane + half / 8 : lane - half / 8);
    float c[8], s[8];

    if (ROTATE && (int)blockIdx.y < a.q_chunks) {
        // ---- query heads: rotate into q_out ----
        const int g0 = blockIdx.y * a.rounds * kIter;   // first group of heads
        const __half *src = a.q + token * a.q_stride + (int64_t)g0 * group_dim + within;
        __half *dst = a.q_out + token * a.num_q_heads * head_dim + (int64_t)g0 * group_dim + within;
        const int left = live ? a.num_q_heads - g0 * hpw - sub : 0;   // head i * hpw exists while i * hpw < left
#pragma unroll 1
        for (int r = 0; r < a.rounds; ++r) {
            uint4 raw[kIter];
#pragma unroll
            for (int i = 0; i < kIter; ++i)
                if ((r * kIter + i) * hpw < left) raw[i] = *reinterpret_cast<const uint4 *>(src + i * group_dim);
            if (r == 0) {
                if (!pos_ok) {                          // the same on every lane
                    if (blockIdx.y == 0 && lane == 0) report(a.err_flag, KVQ_DEV_BAD_POS);
                    return;
                }
                if (turns) load_turn(a, pos, ch, c, s);
            }
#pragma unroll
            for (int i = 0; i < kIter; ++i) {
                uint4 other = raw[i];
                if (!a.interleaved) other = shuffle4(raw[i], mate);
                if (turns) {
                    float x[8];
                    unpack8(raw[i], x);
                    rotate8(x, other, a.interleaved, c, s);
                    raw[i] = pack8(x);
                }
                if ((r * kIter + i) * hpw < left) *reinterpret_cast<uint4 *>(dst + i * group_dim) = raw[i];
            }
            src += kIter * group_dim;
            dst += kIter * group_dim;
        }
        return;
    }

    // ---- key heads (rotated), then value heads, into the pools ----
    const int32_t slot = __ldg(a.slots + token);
    const int64_t page = slot >> 2;
    const bool keep = slot >= 0 && page < a.num_pages;
    const int chunk = blockIdx.y - (ROTATE ? a.q_chunks : 0);
    if (lane == 0 && chunk == 0) {
        if (!pos_ok && a.q_chunks == 0) report(a.err_flag, KVQ_DEV_BAD_POS);
        if (pos_ok && slot >= 0 && !keep) report(a.err_flag, KVQ_DEV_BAD_SLOT);
    }
    if (!keep || !pos_ok) return;                       // the same on every lane
    const int groups = (a.num_kv_heads + hpw - 1) / hpw;   // groups of key heads, and of value heads
    const __half *ksrc = a.k + token * a.k_stride + within, *vsrc = a.v + token * a.v_stride + within;
    const int64_t unit0 = page * a.num_kv_heads;        // (page, kv head 0)
#pragma unroll 1
    for (int r = 0; r < a.rounds; ++r) {
        const int g0 = (chunk * a.rounds + r) * kIter;
        uint4 raw[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int gi = g0 + i;
            const bool is_v = gi >= groups;
            const int g = is_v ? gi - groups : gi;
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live && g < groups && g * hpw + sub < a.num_kv_heads)
                raw[i] = *reinterpret_cast<const uint4 *>((is_v ? vsrc : ksrc) + g * group_dim);
        }
        if (turns && g0 < groups) load_turn(a, pos, ch, c, s);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int gi = g0 + i;
            if (gi >= 2 * groups) break;                // the same on every lane
            const bool is_v = gi >= groups;
            const int h = (is_v ? gi - groups : gi) * hpw + sub;
            const bool mine = live && h < a.num_kv_heads;
            float x[8];
            unpack8(raw[i], x);
            if (ROTATE && !is_v) {
                uint4 other = raw[i];
                if (!a.interleaved) other = shuffle4(raw[i], mate);
                if (turns) {
                    rotate8(x, other, a.interleaved, c, s);
                    if (POOL == PoolKind::fp16) raw[i] = pack8(x);
                }
            }
            uint8_t *pool = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache);
            const float scale = is_v ? a.v_scale : a.k_scale;
            if constexpr (POOL == PoolKind::e2m1) {
                // the block of 16: this lane's eight channels and its neighbour's
                uint32_t m = absmax8_bits(x);
                m = max(m, __shfl_xor_sync(kAll, m, 1));
                if (!mine) continue;
                const E2m1Block blk = e2m1_block(m, is_v ? a.v_six : a.k_six, scale);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], blk.factor);
                uint8_t *dst = pool + (unit0 + h) * e2m1_page_bytes(head_dim);
                *reinterpret_cast<uint32_t *>(dst + (slot & 3) * (head_dim / 2) + ch / 2) = e2m1_pack8(x);
                if ((vec & 1) == 0) dst[e2m1_scale_off(head_dim) + (ch / 16) * 4 + (slot & 3)] = (uint8_t)blk.scale;
            } else if (mine) {
                const int64_t at = ((unit0 + h) * 4 + (slot & 3)) * head_dim + ch;
                if constexpr (POOL == PoolKind::e4m3)
                    *reinterpret_cast<uint2 *>(pool + at) = quantize8(x, scale);
                else
                    *reinterpret_cast<uint4 *>(pool + 2 * at) = raw[i];
            }
        }
    }
}

template <PoolKind POOL, bool ROTATE>
static cudaError_t launch_append_rope_dim(dim3 grid, const RopeArgs &a, cudaStream_t stream)
{
    const dim3 block(kRopeThreads);
    if (a.head_dim == 128) return launch_pdl(append_rope_kernel<POOL, ROTATE, 128>, grid, block, 0, stream, a);
    if (a.head_dim == 64) return launch_pdl(append_rope_kernel<POOL, ROTATE, 64>, grid, block, 0, stream, a);
    if constexpr (POOL != PoolKind::e2m1)
        return launch_pdl(append_rope_kernel<POOL, ROTATE, 0>, grid, block, 0, stream, a);
    return cudaErrorInvalidValue;
}

cudaError_t launch_append_rope(PoolKind pool, bool rotate, RopeArgs a, cudaStream_t stream)
{
    if (a.num_tokens == 0) return cudaSuccess;
    const int hpw = 32 / (a.head_dim / 8);
    // one round of kIter groups a warp while the warps are few, up to two where they fill the card
    a.rounds = (int64_t)a.num_tokens * (a.num_q_heads + 2 * a.num_kv_heads) > (int64_t)device_sm_count() * 64 * 2 * kIter * hpw ? 2 : 1;
    const int per = a.rounds * kIter * hpw;   // heads of a warp
    a.q_chunks = (a.num_q_heads + per - 1) / per;
    const int kv_chunks = (2 * ((a.num_kv_heads + hpw - 1) / hpw) + a.rounds * kIter - 1) / (a.rounds * kIter);
    const dim3 grid((unsigned)((a.num_tokens + kRopeThreads / 32 - 1) / (kRopeThreads / 32)), (unsigned)(a.q_chunks + kv_chunks));
    if (grid.y > 65535u) return cudaErrorInvalidConfiguration;
    if (!rotate) return launch_append_rope_dim<PoolKind::e2m1, false>(grid, a, stream);
    if (pool == PoolKind::e2m1) return launch_append_rope_dim<PoolKind::e2m1, true>(grid, a, stream);
    if (pool == PoolKind::e4m3) return launch_append_rope_dim<PoolKind::e4m3, true>(grid, a, stream);
    return launch_append_rope_dim<PoolKind::fp16, true>(grid, a, stream);
}

// ---------------------------------------------------------------------------
// Read-back: the rows of the listed slots as fp16, fl16(fl32(E2M1 * b) * S);
// E2M1 * b has at most 6 significant bits, so the product with S is the only
// binary32 rounding.  A lane owns 8 channels, a warp whole heads of one token's
// K and then V, kIter groups of them loaded before any is stored.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) gather_e2m1_kernel(const uint8_t *__restrict__ k_cache,
                                                                   const uint8_t *__restrict__ v_cache, int64_t num_pages,
                                                                   const int32_t *__restrict__ slots, int num_tokens,
                                                                   int num_kv_heads, float k_scale, float v_scale,
                                                                   __half *__restrict__ k_out, __half *__restrict__ v_out,
                                                                   int32_t *err_flag)
{
    constexpr int lanes = D / 8, hpw = 32 / lanes;
    grid_dependency_wait();   // the preceding kernel may write the pools
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t token = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (token >= num_tokens) return;
    const int sub = lane / lanes, vec = lane % lanes;
    const int32_t slot = __ldg(slots + token);
    const int64_t page = slot >> 2;
    const bool held = slot >= 0 && page < num_pages;      // the same on every lane
    if (slot >= 0 && !held && lane == 0 && blockIdx.y == 0) report(err_flag, KVQ_DEV_BAD_SLOT);
    const int groups = (num_kv_heads + hpw - 1) / hpw;    // groups of key heads, and of value heads
    const int g0 = blockIdx.y * kIter;
    uint32_t code[kIter];
    uint32_t scale[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const bool is_v = g0 + i >= groups;
        const int h = (is_v ? g0 + i - groups : g0 + i) * hpw + sub;
        code[i] = scale[i] = 0u;
        if (held && h < num_kv_heads) {
            const uint8_t *src = (is_v ? v_cache : k_cache) + (page * num_kv_heads + h) * e2m1_page_bytes(D);
            code[i] = __ldg(reinterpret_cast<const uint32_t *>(src + (slot & 3) * (D / 2)) + vec);
            scale[i] = __ldg(src + e2m1_scale_off(D) + (vec / 2) * 4 + (slot & 3));
        }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const bool is_v = g0 + i >= groups;
        const int h = (is_v ? g0 + i - groups : g0 + i) * hpw + sub;
        if (h >= num_kv_heads) continue;                  // (a group past the last value head as well)
        const float block = e4m3_value(scale[i]), layer = is_v ? v_scale : k_scale;
        const uint32_t p[4] = {e2m1_pair<0>(code[i]), e2m1_pair<1>(code[i]), e2m1_pair<2>(code[i]), e2m1_pair<3>(code[i])};
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p[j]));
            y[2 * j] = __fmul_rn(__fmul_rn(f.x, block), layer);
            y[2 * j + 1] = __fmul_rn(__fmul_rn(f.y, block), layer);
        }
        *reinterpret_cast<uint4 *>((is_v ? v_out : k_out) + (token * num_kv_heads + h) * D + vec * 8) = pack8(y);
    }
}

template <int D>
static cudaError_t launch_gather_dim(const void *k_cache, const void *v_cache, int64_t num_pages, const int32_t *slots,
                                     int32_t num_tokens, int32_t num_kv_heads, float k_scale, float v_scale, void *k_out,
                                     void *v_out, int32_t *err_flag, cudaStream_t stream)
{
    constexpr int hpw = 32 / (D / 8);
    const int groups = 2 * ((num_kv_heads + hpw - 1) / hpw);
    const dim3 grid((unsigned)((num_tokens + kRopeThreads / 32 - 1) / (kRopeThreads / 32)), (unsigned)((groups + kIter - 1) / kIter));
    if (grid.y > 65535u) return cudaErrorInvalidConfiguration;
    return launch_pdl(gather_e2m1_kernel<D>, grid, dim3(kRopeThreads), 0, stream, static_cast<const uint8_t *>(k_cache),
                      static_cast<const uint8_t *>(v_cache), num_pages, slots, num_tokens, num_kv_heads, k_scale, v_scale,
                      static_cast<__half *>(k_out), static_cast<__half *>(v_out), err_flag);
}

cudaError_t launch_gather_e2m1(const void *k_cache, const void *v_cache, int64_t num_pages, const int32_t *slots,
                               int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
                               void *k_out, void *v_out, int32_t *err_flag, cudaStream_t stream)
{
    if (num_tokens == 0) return cudaSuccess;
    return head_dim == 128 ? launch_gather_dim<128>(k_cache, v_cache, num_pages, slots, num_tokens, num_kv_heads, k_scale,
                                                    v_scale, k_out, v_out, err_flag, stream)
                           : launch_gather_dim<64>(k_cache, v_cache, num_pages, slots, num_tokens, num_kv_heads, k_scale,
                                                   v_scale, k_out, v_out, err_flag, stream);
}

// ---------------------------------------------------------------------------
// The rotation table, one thread per (position, pair): angles in binary64 (at
// position 262,143 a binary32 angle is off by up to 2^-7 radians), rounded to
// binary32 after cos and sin.  Made once when a model is loaded.
__global__ void __launch_bounds__(256) rope_table_kernel(float *__restrict__ table, int32_t max_positions, int32_t half,
                                                         double base, int32_t kind, double factor, double low, double high,
                                                         double magnitude)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (int64_t)max_positions * half) return;
    const int64_t p = i / half;
    const int j = (int)(i - p * half);
    double f = pow(base, -(double)j / half);
    if (kind == KVQ_ROPE_LINEAR) f /= factor;
    if (kind == KVQ_ROPE_YARN) {
        const double ramp = fmin(fmax((j - low) / (high - low), 0.0), 1.0);
        f = f / factor * ramp + f * (1.0 - ramp);
    }
    double sn, cs;
    sincos((double)p * f, &sn, &cs);
    table[p * 2 * half + j] = (float)(cs * magnitude);
    table[p * 2 * half + half + j] = (float)(sn * magnitude);
}

cudaError_t launch_rope_table(float *table, int32_t max_positions, int32_t rot_dim, double base, int32_t kind, double factor,
                              double low, double high, double magnitude, cudaStream_t stream)
{
    const int64_t n = (int64_t)max_positions * (rot_dim / 2);
    const int64_t blocks = (n + 255) / 256;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    rope_table_kernel<<<(unsigned)blocks, 256, 0, stream>>>(table, max_positions, rot_dim / 2, base, kind, factor, low, high,
                                                            magnitude);
    return cudaGetLastError();
}

}  // namespace kvq
