// gated.cu -- the gated feed-forward block on rows grouped by expert: both projections, the activation and
// the product in one kernel, and the way back through the down projection and the activation:
//   forward   g = Wg_e x, u = Wu_e x, h = act(g) u;              g and u may be kept for the backward pass
//   dgrad     dh = Wd_e^T dy, dg = dh u act'(g), du = dh act(g), h = act(g) u again; g and u as kept
// Both are the products of gemm.cuh with other epilogues.
#include "checkpoint.cuh"
#include "gemm.cuh"

namespace ep {
namespace {

// ------------------------------------------------------------------ activation

// act(g) = g s(z), s the logistic function: silu z = g; gelu (the form with a hyperbolic tangent)
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3). For gelu z is taken at |g| <= 16, beyond which s is 0 or 1 in
// fp32 and g^3 could overflow.
struct Activated {
    float value, slope;
};
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }
constexpr float kGelu = 1.5957691216057308f, kCubic = 0.044715f;
template <int ACT>
__device__ __forceinline__ float gate_slope_at(float& z, float g) {          // z, and its slope
    if (ACT == EP_ACT_SILU) {
        z = g;
        return 1.0f;
    }
    const float t = fminf(fmaxf(g, -16.0f), 16.0f), t2 = t * t;
    z = kGelu * t * fmaf(kCubic, t2, 1.0f);
    return kGelu * fmaf(3.0f * kCubic, t2, 1.0f);
}
template <int ACT>
__device__ __forceinline__ float activate(float g) {
    float z;
    gate_slope_at<ACT>(z, g);
    return g * logistic(z);
}
template <int ACT>
__device__ __forceinline__ Activated activate_both(float g) {
    float z;
    const float dz = gate_slope_at<ACT>(z, g), s = logistic(z), v = g * s;
    return {v, ACT == EP_ACT_SILU ? fmaf(v, 1.0f - s, s) : fmaf(v * (1.0f - s), dz, s)};
}

// ------------------------------------------------------------------ what is kept

// g and u of a row: bf16 [rows][2][F], or e4m3 [rows][2][F padded to 16] with a byte for each 16
// features, [rows][groups][2], so that a row's 64 or 128 features of a tile have theirs in 8 or 16 bytes.
enum Keep { kNone, kBf16, kE4m3 };

struct Kept {
    void* values;
    uint8_t* scales;
    int F, padded;
    __device__ __forceinline__ __nv_bfloat16* halves(int64_t row, int side) const {
        return reinterpret_cast<__nv_bfloat16*>(values) + (2 * row + side) * F;
    }
    __device__ __forceinline__ uint8_t* bytes(int64_t row, int side) const {
        return reinterpret_cast<uint8_t*>(values) + (2 * row + side) * padded;
    }
    __device__ __forceinline__ uint8_t* exponent(int64_t row, int side, int feature) const {
        return scales + (row * (padded / kKeptGroup) + feature / kKeptGroup) * 2 + side;
    }
};

// ------------------------------------------------------------------ forward

// Four warps, one for each quarter of the lanes, bring the same rows of a tile into the order of memory in
// shared memory that they have together: a warp alone has 32 bytes of a row of h, which cost the way to L2
// a request each, all four have its whole 128 bytes.
__device__ __forceinline__ void quarters_barrier(int part) { asm volatile("bar.sync %0, 128;" ::"r"(2 + part) : "memory"); }

// The M side has eight rows of Wg and eight of Wu in turn, so that a warp has both sums of a feature
// in the same place of two sets of eight lanes, and a tile of 256 covers 128 features.
template <Keep KEEP, int ACT>
struct Gated : NoExtra {
    static constexpr bool kPairs = true, kWrites = true;
    static constexpr int kStaged = 4096, kFloats = kWarps * kStaged / 16, kFewFloats = kFloats;          // kStaged: of four warps
    Kept kept;
    __device__ __forceinline__ void tile(uint32_t tmem, float* shared, unsigned char*, __nv_bfloat16* out, int64_t row0, int rows,
                                         int m0, int M, int half, int lane) const {
        write<kWarps / 4>(tmem, smem_addr(shared), out, row0, rows, m0, M, half, lane);
    }
    __device__ __forceinline__ void prefetch(int64_t, int, int, int, int) const {}

    // 64 features x 32 rows at a time, 16 features of blocks b of 8 rows a warp. Lane 4g + c has rows 2c, 2c+1 of
    // features 8t + g of each block; afterwards it has chunk lane & 7 (eight features) of rows lane / 8 and 4 +
    // lane / 8 of its quarter of the rows. Chunk n of row r is at r * 128 + (n ^ (r & 7)) * 16, where neither
    // direction meets in a bank. (Exchanging registers between lanes instead took twice the instructions.)
    static __device__ __forceinline__ void by_rows(const uint32_t (&p)[2][4], uint32_t stage, int part, int quarter, int lane, uint4 (&q)[2]) {
        quarters_barrier(part);          // what was there has been read
#pragma unroll
        for (int t = 0; t < 2; ++t) store_blocks(stage + lane * 128 + (((quarter * 2 + t) ^ (lane & 7)) << 4), p[t]);
        quarters_barrier(part);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = quarter * 8 + j * 4 + (lane >> 3);
            q[j] = ld_shared_v4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
    }
    template <int PARTS>          // how many sets of four warps share the rows
    __device__ __forceinline__ void write(uint32_t tmem, uint32_t stage, __nv_bfloat16* out, int64_t row0, int rows, int m0, int M,
                                          int part, int lane) const {
        const int F = M / 2, quarter = (threadIdx.x >> 5) & 3, f0 = m0 / 2 - quarter * 16, f = f0 + (lane & 7) * 8;
        if (f0 >= F) return;
        stage += part * kStaged;
        for (int n = part * 32; n < rows; n += PARTS * 32) {
            float v[4][2][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                tmem_load_16x8(tmem + n + b * 8, v[b][0]);
                tmem_load_16x8(tmem + n + b * 8 + (16u << 16), v[b][1]);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_wait(v[b]);
            const int64_t row = row0 + n + quarter * 8 + (lane >> 3);
            const int left = rows - n - quarter * 8 - (lane >> 3);          // of the rows from that one on
            uint32_t p[2][4];
            uint4 q[2];
            if (out != nullptr) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        p[t][b] = pack_bf16x2(activate<ACT>(v[b][t][0]) * v[b][t][2], activate<ACT>(v[b][t][1]) * v[b][t][3]);
                by_rows(p, stage, part, quarter, lane, q);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j * 4 < left && f < F) st_v4(out + (row + j * 4) * F + f, q[j]);
            }
            uint32_t exponent[2][2];          // by side, row
#pragma unroll
            for (int h = 0; h < (KEEP == kNone ? 0 : 2); ++h) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int t = 0; t < 2; ++t) p[t][b] = pack_bf16x2(v[b][t][2 * h], v[b][t][2 * h + 1]);
                by_rows(p, stage, part, quarter, lane, q);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (KEEP == kBf16) {
                        if (j * 4 < left && f < F) st_v4(kept.halves(row + j * 4, h) + f, q[j]);
                        continue;
                    }
                    // The group is this lane's eight features and its neighbour's.
                    uint32_t m = larger_bf16x2(magnitudes(q[j].x), magnitudes(q[j].y));
                    m = larger_bf16x2(m, larger_bf16x2(magnitudes(q[j].z), magnitudes(q[j].w)));
                    m = larger_bf16x2(m, __byte_perm(m, 0, 0x1032));
                    m = larger_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                    const uint32_t e = exponent[h][j] = kept_exponent(larger_bf16x2(m, 0) & 0xFFFFu);          // 0: nothing but NaN
                    const float inv = kept_inverse(e);
                    uint2 eight = make_uint2(keep_pair(q[j].x, inv) | keep_pair(q[j].y, inv) << 16,
                                             keep_pair(q[j].z, inv) | keep_pair(q[j].w, inv) << 16);
                    if (f >= F) eight = make_uint2(0, 0);          // padding: an infinite row's sums are NaN there
                    if (j * 4 < left && f < kept.padded) *reinterpret_cast<uint2*>(kept.bytes(row + j * 4, h) + f) = eight;
                }
            }
            if (KEEP == kE4m3 && (lane & 1) == 0 && f < kept.padded)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j * 4 < left)
                        *reinterpret_cast<uint16_t*>(kept.exponent(row + j * 4, 0, f)) = (uint16_t)(exponent[0][j] | exponent[1][j] << 8);
        }
    }
};

// Sixteen warps write where the writing takes longer than a tile's products (more of them that wait slow the
// warps that issue). Keeping 8 bits, 8 and 16 warps: 17107 rows 312 -> 2688 107 and 90 us, 4229 rows 560 -> 2616
// 39.5 and 36.0, 2048 rows 2048 -> 1024 34.7 and 35.5.
constexpr int kShort = 12 * kBK;          // contractions up to here
template <Keep KEEP, int ACT>
struct GatedShort : Gated<KEEP, ACT> {
    using Base = Gated<KEEP, ACT>;
    static constexpr int kWarps = 16, kFloats = kWarps * Base::kStaged / 16;
    __device__ __forceinline__ void tile(uint32_t tmem, float* shared, unsigned char*, __nv_bfloat16* out, int64_t row0, int rows,
                                         int m0, int M, int half, int lane) const {
        Base::template write<kWarps / 4>(tmem, smem_addr(shared), out, row0, rows, m0, M, half, lane);
    }
};

// ------------------------------------------------------------------ single tokens

// One row, nothing kept: a stream of its expert's weights past it without tensor cores, whose set-up and
// joining of parts are what such a call takes longest (1 row 4096 -> 4096: 15.4 us by gemm_split_kernel, so
// 12.5; 1024 -> 1024 6.9, 2.7; two rows and more are as fast by tensor cores). Small blocks that ask
// for all of their weights at once and leave: with many of them an SM 64 MB come in 10.7 us, where blocks that
// stay and load ahead take 12.5. `team` warps have a feature's two rows of weights, AHEAD pieces of 16
// bytes a thread and row at a time. fp32 sums: a thread's, of even and of odd values, then over the lanes,
// then over the team's warps in order.
constexpr int kTokenThreads = 256, kTokenWarps = kTokenThreads / 32;
struct TokenArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* w;
    const int32_t* prefix;
    __nv_bfloat16* h;
    uint32_t* err;
    int E, K, F, act;
    int team;          // 1, 2, 4 or 8
};

// A bf16 pair as two fp32 values, and two multiply-adds at once.
__device__ __forceinline__ uint64_t wide_pair(uint32_t w) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(w << 16), "r"(w & 0xFFFF0000u));
    return r;
}
__device__ __forceinline__ void add_products(uint64_t& sum, const uint4& a, const uint4& b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(wide_pair(x[i])), "l"(wide_pair(y[i])));
}

template <int AHEAD>
__global__ void __launch_bounds__(kTokenThreads, AHEAD == 2 ? 6 : 4) token_kernel(const TokenArgs a) {
    __shared__ int s_expert;
    __shared__ float s_sum[kTokenWarps][2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int in = warp & (a.team - 1), f = (int)blockIdx.x * (kTokenWarps / a.team) + warp / a.team;
    const int width = a.team * 256, k_first = in * 256 + lane * 8;
    const int64_t up = (int64_t)a.F * a.K;
    uint4 q[AHEAD][2];
    auto load = [&](int expert, int k0) {
        const __nv_bfloat16* w = a.w + ((int64_t)expert * 2 * a.F + f) * a.K;
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            const int k = k0 + d * width;
            if (f < a.F && k < a.K) {
                q[d][0] = ld_stream_v4(w + k);
                q[d][1] = ld_stream_v4(w + up + k);
            }
        }
    };
    if (threadIdx.x == 0) s_expert = -1;
    pdl_wait();
    if (a.E == 1) load(0, k_first);          // (its weights are these whether or not it has the row)
    __syncthreads();
    bool bad = false;
    for (int e = threadIdx.x; e < a.E; e += kTokenThreads) {
        const int begin = a.prefix[e], end = a.prefix[e + 1];
        bad |= begin < 0 || end > 1 || end < begin;
        if (begin <= 0 && end >= 1) s_expert = e;
    }
    if (bad && blockIdx.x == 0) raise_flag(a.err, EP_DEVERR_RECV_OVERFLOW);
    __syncthreads();
    const int expert = s_expert;
    if (expert >= 0) {
        if (a.E > 1) load(expert, k_first);
        uint64_t sum[2] = {};
        for (int k0 = k_first;;) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int k = k0 + d * width;
                if (f >= a.F || k >= a.K) break;
                const uint4 x = *reinterpret_cast<const uint4*>(a.x + k);
                add_products(sum[0], q[d][0], x);
                add_products(sum[1], q[d][1], x);
            }
            k0 += AHEAD * width;
            if (k0 - k_first >= a.K) break;
            load(expert, k0);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v = __uint_as_float((uint32_t)sum[h]) + __uint_as_float((uint32_t)(sum[h] >> 32));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) s_sum[warp][h] = v;
        }
        __syncthreads();
        if (in == 0 && lane == 0 && f < a.F) {
            float g = 0.0f, u = 0.0f;
            for (int i = 0; i < a.team; ++i) {
                g += s_sum[warp + i][0];
                u += s_sum[warp + i][1];
            }
            a.h[f] = __float2bfloat16_rn((a.act == EP_ACT_SILU ? activate<EP_ACT_SILU>(g) : activate<EP_ACT_GELU_TANH>(g)) * u);
        }
    }
    pdl_trigger();
}

// ------------------------------------------------------------------ backward

struct Back {
    __nv_bfloat16* dgu;          // [rows][2][F]
    __nv_bfloat16* h;            // [rows][F], NULL to leave out
};

// The sums are dh. What was kept is read by rows, eight features a lane, and comes into the sums' layout by way
// of shared memory, as the results come out of it (its values are exact in bf16).
template <Keep KEEP, int ACT>
struct GatedBack : NoExtra {
    static constexpr bool kWrites = true;
    static constexpr int kWarps = 16, kBlock = 2048, kStaged = 3 * kBlock, kFloats = kWarps * kStaged / 16, kFewFloats = kFloats / 2;
    Kept kept;
    Back to;
    // Eight features of one row's side as they are stored, and as four bf16 pairs.
    struct Raw {
        uint4 q;          // e4m3: two words, and the power of two's byte in the third
    };
    __device__ __forceinline__ Raw load(int64_t row, int side, int f) const {
        if constexpr (KEEP == kBf16) return {ld_stream_v4(kept.halves(row, side) + f)};
        uint2 q;
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(kept.bytes(row, side) + f));
        return {make_uint4(q.x, q.y, __ldg(kept.exponent(row, side, f)), 0)};
    }
    static __device__ __forceinline__ uint4 pairs(const Raw& r) {
        if constexpr (KEEP == kBf16) return r.q;
        const float s = kept_scale(r.q.z);
        return make_uint4(kept_pair(r.q.x, s), kept_pair(r.q.x >> 16, s), kept_pair(r.q.y, s), kept_pair(r.q.y >> 16, s));
    }
    __device__ __forceinline__ void prepare(float*, unsigned char*, int64_t row0, int rows, int m0) const {
        prefetch(row0, rows, m0, threadIdx.x - 128, 32 * kWarps);
    }
    // What was kept of a tile, towards L2 while its products run: 128 features of both sides.
    __device__ __forceinline__ void prefetch(int64_t row0, int rows, int m0, int thread, int threads) const {
        const int bytes = KEEP == kBf16 ? 2 : 1, width = min(128, kept.F - m0) * bytes;
        for (int i = thread; i < rows * 2; i += threads) {
            const char* at = KEEP == kBf16 ? reinterpret_cast<const char*>(kept.halves(row0 + (i >> 1), i & 1) + m0)
                                           : reinterpret_cast<const char*>(kept.bytes(row0 + (i >> 1), i & 1) + m0);
            for (int o = 0; o < width; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + o));
        }
    }
    __device__ __forceinline__ void tile(uint32_t tmem, float* shared, unsigned char*, __nv_bfloat16* out, int64_t row0, int rows, int m0,
                                         int M, int half, int lane) const {
        write<kWarps / 4>(tmem, smem_addr(shared), out, row0, rows, m0, M, half, lane);
    }
    // 128 features x 8 rows at a time, 32 features a warp; the next rows' loads are under way meanwhile. In shared
    // memory chunk n (eight features) of row r is at r * 256 + (n ^ r) * 16, where neither direction meets in a
    // bank; a lane reads and writes chunk lane & 15 of row lane / 16 of its quarter of the rows.
    template <int PARTS>
    __device__ __forceinline__ void write(uint32_t tmem, uint32_t stage, __nv_bfloat16*, int64_t row0, int rows, int m0, int M, int part,
                                          int lane) const {
        const int quarter = (threadIdx.x >> 5) & 3, r = quarter * 2 + (lane >> 4), f = m0 - quarter * 32 + (lane & 15) * 8;
        if (m0 - quarter * 32 >= M) return;
        stage += part * kStaged;
        const uint32_t by_row = stage + r * 256 + (((lane & 15) ^ r) << 4);
        const uint32_t by_block = stage + (lane & 7) * 256 + (((quarter * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
        Raw next[2] = {};
        if (part * 8 + r < rows && f < M)
#pragma unroll
            for (int h = 0; h < 2; ++h) next[h] = load(row0 + part * 8 + r, h, f);
        for (int n = part * 8; n < rows; n += 8 * PARTS) {
            const bool there = n + r < rows && f < M;
            const int64_t row = row0 + n + r;
            float v[2][4];
            tmem_load_16x8(tmem + n, v[0]);
            tmem_load_16x8(tmem + n + (16u << 16), v[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) st_shared_v4(by_row + h * kBlock, pairs(next[h]));
            quarters_barrier(part);
            if (n + 8 * PARTS + r < rows && f < M)
#pragma unroll
                for (int h = 0; h < 2; ++h) next[h] = load(row + 8 * PARTS, h, f);
            uint32_t side[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) load_blocks(by_block + h * kBlock, side[h]);
            tmem_wait(v);
            uint32_t p[3][4];          // dg, du, h
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float d0 = v[i >> 1][(i & 1) * 2], d1 = v[i >> 1][(i & 1) * 2 + 1];
                const float u0 = bf16_lo(side[1][i]), u1 = bf16_hi(side[1][i]);
                const Activated a0 = activate_both<ACT>(bf16_lo(side[0][i])), a1 = activate_both<ACT>(bf16_hi(side[0][i]));
                p[0][i] = pack_bf16x2(d0 * u0 * a0.slope, d1 * u1 * a1.slope);
                p[1][i] = pack_bf16x2(d0 * a0.value, d1 * a1.value);
                p[2][i] = pack_bf16x2(a0.value * u0, a1.value * u1);
            }
            // A warp's blocks of what was kept are its own blocks of the results.
#pragma unroll
            for (int h = 0; h < 3; ++h) store_blocks(by_block + h * kBlock, p[h]);
            quarters_barrier(part);
            uint4 q[3];
#pragma unroll
            for (int h = 0; h < 3; ++h) q[h] = ld_shared_v4(by_row + h * kBlock);
            if (there) {
                st_v4(to.dgu + 2 * row * M + f, q[0]);
                st_v4(to.dgu + (2 * row + 1) * M + f, q[1]);
                if (to.h != nullptr) st_v4(to.h + row * M + f, q[2]);
            }
        }
    }
};

// ------------------------------------------------------------------ host

ep_status check_block(const ep_gemm_shape* sh, const void* rows_in, const void* w, const int32_t* prefix, int32_t act,
                      const ep_launch* launch) {
    if (launch == nullptr || (act != EP_ACT_SILU && act != EP_ACT_GELU_TANH)) return EP_ERR_INVALID_ARG;
    const ep_status st = check_gemm_shape(sh);
    if (st != EP_OK) return st;
    if (prefix == nullptr || ((uintptr_t)prefix & 3) != 0) return EP_ERR_INVALID_ARG;
    if (sh->num_rows > 0 && (rows_in == nullptr || w == nullptr)) return EP_ERR_INVALID_ARG;
    return (((uintptr_t)rows_in | (uintptr_t)w) & 15) != 0 ? EP_ERR_INVALID_ARG : EP_OK;
}

// A checkpoint of g and u: a row's two bytes of scales are written together.
ep_status check_sides(const ep_checkpoint* c, bool rows) {
    const ep_status st = check_checkpoint(c, rows, true);
    return st == EP_OK && ((uintptr_t)c->scales & 1) != 0 ? EP_ERR_INVALID_ARG : st;
}

Kept kept_of(const ep_checkpoint* c, int F) {
    Kept k{nullptr, nullptr, F, kept_features(F)};
    if (c != nullptr) k.values = c->values, k.scales = c->scales;
    return k;
}

template <Direction D, class Wide, class Few>
ep_status run_block(const GemmMaps& maps, const GemmArgs& a, const Wide& wide, const Few& few, cudaStream_t stream) {
    const cudaError_t e = launch_gemm<D>(maps, a, wide, few, stream);
    return e == cudaSuccess ? EP_OK : cuda_fail(e);
}

// Tiles and stages. A pair's tile of 256 x 256 costs 4 us more to set up than two CTAs of 128 x 64, and its epilogue 3
// (forward) to 7 us (backward) that nothing hides in a short call. So tiles are taken that narrow where
//   up to 8 steps of 64 are contracted and four of them are there for each SM (backward six), two being at work,
//   up to 16 and two are there, or where two of 32 rows are, those,
//   up to 32, one and a half are, and experts have 96 rows on average (else tiles of 64 rows read the weights
//   twice where wider ones do so once).
// Wide and so, forward keeping 8 bits / backward, us:
//   509 rows of 8 experts 256 -> 512     9.0 / 10.4    4.5 / 4.8      200 rows of one 2048 -> 1024   13.3 / 14.5   10.0 / 8.1
//   1500 rows of 8 1024 -> 512          14.4 / 17.6    8.5 / 8.8      1200 rows of 8 2048 -> 512     15.1 / 15.9   13.2 / 11.8
//   8191 rows of 32 512 -> 512          29.3 / 31.8   (29.2)/ 20.8    509 rows of 8 2048 -> 1024     18.4 / 12.0  (16.7 / 12.7)
//                                                                     150 rows of one 7168 -> 2048   20.5 / 16.0  (23.2 / 14.9)
void block_tiles(GemmArgs* a, bool back) {
    const int steps = ceil_div(a->C, kBK), sms = sm_count();
    int widest = 256, parts = 8;
    for (int bn = 64; bn >= 32; bn /= 2) {
        a->bn = bn;
        const int64_t tiles = gemm_most_tiles(*a, false, kBM);
        int halves = steps <= 16 ? 4 : 0;          // of the SMs
        if (bn == 64 && steps <= 8) halves = back ? 12 : 8;
        if (bn == 64 && steps > 16 && steps <= 32 && a->num_rows / 96 >= a->E) halves = 3;
        if (2 * tiles > (int64_t)halves * sms) continue;
        widest = bn;
        parts = tiles > sms ? 1 : 8;          // (gemm_tiles' own count of the tiles is the least there can be)
    }
    gemm_tiles(a, false, 0, 256, widest, 16, parts);
}

// The maps of the rows, in boxes of a.box, and for gemm_kernel of twice that.
ep_status encode_rows(GemmMaps* maps, const GemmArgs& a, const void* rows) {
    const uint64_t d[2] = {(uint64_t)a.C, (uint64_t)a.num_rows};
    uint32_t box[2] = {64, (uint32_t)a.box};
    const ep_status st = encode_map(&maps->b, rows, 2, d, box);
    if (st != EP_OK || gemm_by_split(a)) return st;
    box[1] *= 2;
    return encode_map(&maps->b2, rows, 2, d, box);
}

template <Keep KEEP, int ACT>
ep_status forward(const GemmMaps& maps, const GemmArgs& a, const Kept& kept, cudaStream_t stream) {
    Gated<KEEP, ACT> extra;
    extra.kept = kept;
    if constexpr (KEEP == kE4m3) {
        GatedShort<KEEP, ACT> wide;
        wide.kept = kept;
        if (a.C <= kShort) return run_block<kForward>(maps, a, wide, extra, stream);
    }
    return run_block<kForward>(maps, a, extra, extra, stream);
}
template <Keep KEEP>
ep_status forward(const GemmMaps& maps, const GemmArgs& a, int act, const Kept& kept, cudaStream_t stream) {
    return act == EP_ACT_SILU ? forward<KEEP, EP_ACT_SILU>(maps, a, kept, stream)
                              : forward<KEEP, EP_ACT_GELU_TANH>(maps, a, kept, stream);
}

template <Keep KEEP, int ACT>
ep_status backward(const GemmMaps& maps, const GemmArgs& a, const Kept& kept, const Back& to, cudaStream_t stream) {
    GatedBack<KEEP, ACT> extra;
    extra.kept = kept;
    extra.to = to;
    return run_block<kDgrad>(maps, a, extra, extra, stream);
}
template <Keep KEEP>
ep_status backward(const GemmMaps& maps, const GemmArgs& a, int act, const Kept& kept, const Back& to, cudaStream_t stream) {
    return act == EP_ACT_SILU ? backward<KEEP, EP_ACT_SILU>(maps, a, kept, to, stream)
                              : backward<KEEP, EP_ACT_GELU_TANH>(maps, a, kept, to, stream);
}

// The calls; `loads` and `wait_ns` as in GemmArgs, for the self-test.
ep_status run_forward(const ep_gemm_shape* sh, const void* x, const void* w, const int32_t* expert_prefix, int32_t activation, void* h,
                      const ep_checkpoint* keep, const ep_launch* launch, int loads, uint64_t wait_ns) {
    ep_status st = check_block(sh, x, w, expert_prefix, activation, launch);
    if (st != EP_OK) return st;
    const bool rows = sh->num_rows > 0;
    if (keep != nullptr && (st = check_sides(keep, rows)) != EP_OK) return st;
    if ((rows && h == nullptr && keep == nullptr) || ((uintptr_t)h & 15) != 0) return EP_ERR_INVALID_ARG;
    if (sh->num_rows == 1 && keep == nullptr && loads == GemmArgs{}.loads) {
        TokenArgs t{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w), expert_prefix,
                    static_cast<__nv_bfloat16*>(h), launch->error_flags, sh->num_experts, sh->in_features, sh->out_features,
                    activation, kTokenWarps};
        // Two pieces of 16 bytes a thread where the block's warps reach that far, else four at a time.
        while (t.team > 1 && t.team * 256 >= t.K) t.team /= 2;
        const dim3 grid((unsigned)(((int64_t)t.F * t.team + kTokenWarps - 1) / kTokenWarps));
        if ((st = begin_call(launch)) != EP_OK) return st;
        const cudaError_t e = launch_pdl(t.K <= kTokenWarps * 512 ? token_kernel<2> : token_kernel<4>, grid, dim3(kTokenThreads), 0,
                                         launch->stream, t);
        return e != cudaSuccess ? cuda_fail(e) : end_call(launch);
    }
    const uint64_t K = (uint64_t)sh->in_features, F = (uint64_t)sh->out_features, E = (uint64_t)sh->num_experts;
    GemmArgs a{};
    a.prefix = expert_prefix;
    a.out = reinterpret_cast<__nv_bfloat16*>(h);
    a.num_rows = sh->num_rows;
    a.E = sh->num_experts;
    a.M = 2 * sh->out_features;
    a.N = a.C = sh->in_features;
    a.err = launch->error_flags;
    a.loads = loads;
    a.wait_ns = wait_ns;
    block_tiles(&a, false);
    GemmMaps maps{};
    if (rows) {
        // Eight rows of Wg, the eight of Wu F rows on, the next eight of both, and so on. (The strides do not
        // ascend: a box's address is a sum over its coordinates, whatever their order.)
        const uint64_t d[5] = {K, 8, 2, F / 8, E}, strides[4] = {2 * K, 2 * F * K, 16 * K, 4 * F * K};
        const uint32_t box[5] = {64, 8, 2, 8, 1};
        if ((st = encode_map(&maps.a, w, 5, d, box, strides)) != EP_OK) return st;
        if ((st = encode_rows(&maps, a, x)) != EP_OK) return st;
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        const Kept kept = kept_of(keep, sh->out_features);
        st = keep == nullptr              ? forward<kNone>(maps, a, activation, kept, launch->stream)
             : keep->dtype == EP_BF16 ? forward<kBf16>(maps, a, activation, kept, launch->stream)
                                          : forward<kE4m3>(maps, a, activation, kept, launch->stream);
        if (st != EP_OK) return st;
    }
    return end_call(launch);
}

ep_status run_backward(const ep_gemm_shape* sh, const void* dy, const void* w, const int32_t* expert_prefix, int32_t activation,
                       const ep_checkpoint* kept, void* dgu, void* h, const ep_launch* launch, int loads, uint64_t wait_ns) {
    ep_status st = check_block(sh, dy, w, expert_prefix, activation, launch);
    if (st != EP_OK) return st;
    const bool rows = sh->num_rows > 0;
    if ((st = check_sides(kept, rows)) != EP_OK) return st;
    if ((rows && dgu == nullptr) || (((uintptr_t)dgu | (uintptr_t)h) & 15) != 0) return EP_ERR_INVALID_ARG;
    GemmArgs a{};
    a.prefix = expert_prefix;
    a.num_rows = sh->num_rows;
    a.E = sh->num_experts;
    a.M = a.N = sh->in_features;
    a.C = sh->out_features;
    a.err = launch->error_flags;
    a.loads = loads;
    a.wait_ns = wait_ns;
    block_tiles(&a, true);
    GemmMaps maps{};
    if (rows) {
        const uint64_t d[3] = {(uint64_t)sh->in_features, (uint64_t)sh->out_features, (uint64_t)sh->num_experts};
        const uint32_t box[3] = {64, 64, 1};
        if ((st = encode_map(&maps.a, w, 3, d, box)) != EP_OK) return st;
        if ((st = encode_rows(&maps, a, dy)) != EP_OK) return st;
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        const Kept k = kept_of(kept, sh->in_features);
        const Back to{reinterpret_cast<__nv_bfloat16*>(dgu), reinterpret_cast<__nv_bfloat16*>(h)};
        st = kept->dtype == EP_BF16 ? backward<kBf16>(maps, a, activation, k, to, launch->stream)
                                    : backward<kE4m3>(maps, a, activation, k, to, launch->stream);
        if (st != EP_OK) return st;
    }
    return end_call(launch);
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status ep_expert_gated(const ep_gemm_shape* sh, const void* x, const void* w, const int32_t* expert_prefix, int32_t activation,
                          void* h, const ep_checkpoint* keep, const ep_launch* launch) {
    return ep::run_forward(sh, x, w, expert_prefix, activation, h, keep, launch, ep::GemmArgs{}.loads, ep::GemmArgs{}.wait_ns);
}

ep_status ep_expert_gated_dgrad(const ep_gemm_shape* sh, const void* dy, const void* w, const int32_t* expert_prefix,
                                int32_t activation, const ep_checkpoint* kept, void* dgu, void* h, const ep_launch* launch) {
    return ep::run_backward(sh, dy, w, expert_prefix, activation, kept, dgu, h, launch, ep::GemmArgs{}.loads, ep::GemmArgs{}.wait_ns);
}

ep_status ep_selftest_gated_timeout(const ep_gemm_shape* sh, int32_t product, const void* rows, const void* w,
                                    const int32_t* expert_prefix, const ep_checkpoint* checkpoint, void* out, int32_t loads,
                                    int32_t timeout_ms, const ep_launch* launch) {
    using namespace ep;
    if (launch == nullptr || launch->error_flags == nullptr || loads < 0 || loads % kBK != 0 || timeout_ms < 1 ||
        timeout_ms > 10000 || product < 0 || product > 1)
        return EP_ERR_INVALID_ARG;
    const uint64_t ns = (uint64_t)timeout_ms * 1000000ull;
    return product == 0 ? run_forward(sh, rows, w, expert_prefix, EP_ACT_SILU, out, checkpoint, launch, loads, ns)
                        : run_backward(sh, rows, w, expert_prefix, EP_ACT_SILU, checkpoint, out, nullptr, launch, loads, ns);
}

}  // extern "C"
