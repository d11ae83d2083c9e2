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
__device__ __forceinline__ float activate(float g, int act) {
    if (act == EP_ACT_SILU) return g * logistic(g);
    const float t = fminf(fmaxf(g, -16.0f), 16.0f);
    return g * logistic(kGelu * (t + kCubic * t * t * t));
}
__device__ __forceinline__ Activated activate_both(float g, int act) {
    if (act == EP_ACT_SILU) {
        const float s = logistic(g);
        return {g * s, s * (1.0f + g * (1.0f - s))};
    }
    const float t = fminf(fmaxf(g, -16.0f), 16.0f), s = logistic(kGelu * (t + kCubic * t * t * t));
    return {g * s, s + g * (s * (1.0f - s)) * (kGelu * (1.0f + 3.0f * kCubic * t * t))};
}

// ------------------------------------------------------------------ what is kept

// g and u of a row: bf16 [rows][2][F], or e4m3 [rows][2][F padded to 16] with a byte for each 16.
enum Keep { kNone, kBf16, kE4m3 };

struct Kept {
    void* values;
    uint8_t* scales;
    int F, padded, act;
    __device__ __forceinline__ __nv_bfloat16* halves(int64_t row, int side) const {
        return reinterpret_cast<__nv_bfloat16*>(values) + (2 * row + side) * F;
    }
    __device__ __forceinline__ uint8_t* bytes(int64_t row, int side) const {
        return reinterpret_cast<uint8_t*>(values) + (2 * row + side) * padded;
    }
    __device__ __forceinline__ uint8_t* exponent(int64_t row, int side, int feature) const {
        return scales + (2 * row + side) * (padded / kKeptGroup) + feature / kKeptGroup;
    }
};

__device__ __forceinline__ void store_half(__nv_bfloat16* at, float v) { *at = __float2bfloat16_rn(v); }

// ------------------------------------------------------------------ forward

// The M side has eight rows of Wg and eight of Wu in turn, so that a warp has both sums of a feature
// in the same place of two sets of eight lanes, and a tile of 256 covers 128 features.
template <Keep KEEP>
struct GatedWide : NoExtra {
    static constexpr bool kPairs = true;
    Kept kept;
    // g and u of those 16 rows; `row` is this lane's.
    __device__ __forceinline__ void keep_block(const float (&v)[2][2][4], int64_t row, bool there, int f0, int F, int c) const {
        uint32_t side[2][4];          // g, u: block b's features 8t + 2c, 2c+1 of row g in 2b + t
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float(&s)[4] = v[i >> 1][i & 1];
            side[0][i] = transpose_8x8(pack_bf16x2(s[0], s[1]));
            side[1][i] = transpose_8x8(pack_bf16x2(s[2], s[3]));
        }
        if constexpr (KEEP == kBf16) {
            const int f = f0 + (c & 1) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 q = transpose_quad(side[h], c);
                if (there && f < F) st_v4(kept.halves(row, h) + f, q);
            }
        } else {
            uint32_t p[4], e[4];          // 2b + h
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t mg = larger_bf16x2(side[0][2 * b], side[0][2 * b + 1]);
                const uint32_t mu = larger_bf16x2(side[1][2 * b], side[1][2 * b + 1]);
                uint32_t m = larger_bf16x2(__byte_perm(mg, mu, 0x5410), __byte_perm(mg, mu, 0x7632));
                m = larger_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = larger_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                e[2 * b] = kept_exponent(m & 0xFFFFu);
                e[2 * b + 1] = kept_exponent(m >> 16);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float inv = kept_inverse(e[2 * b + h]);
                    p[2 * b + h] = keep_pair(side[h][2 * b], inv) | keep_pair(side[h][2 * b + 1], inv) << 16;
                }
            }
            const uint4 q = transpose_quad(p, c);          // lane c: all 16 features of block c / 2, side c & 1
            if (there) {
                st_v4(kept.bytes(row, c & 1) + f0, make_uint4(__byte_perm(q.x, q.y, 0x5410), __byte_perm(q.z, q.w, 0x5410),
                                                              __byte_perm(q.x, q.y, 0x7632), __byte_perm(q.z, q.w, 0x7632)));
                *kept.exponent(row, c & 1, f0) = (uint8_t)(c < 2 ? (c == 0 ? e[0] : e[1]) : (c == 2 ? e[2] : e[3]));
            }
        }
    }
    // 16 features x 16 rows at a time. Lane 4g + c has rows 2c, 2c+1 of features g (t = 0) and 8 + g
    // (t = 1); after the transpositions the four lanes of row g have eight features each of both blocks
    // of rows.
    __device__ __forceinline__ void tile(uint32_t tmem, float*, unsigned char*, __nv_bfloat16* out, int64_t row0, int rows,
                                         int m0, int M, int half, int lane) const {
        const int g = lane >> 2, c = lane & 3, F = M / 2, f0 = m0 / 2;
        if (f0 >= F) return;
        const int f = f0 + (c & 1) * 8, at = (c >> 1) * 8 + g;
        for (int n = half * 16; n < rows; n += 32) {
            float v[2][2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tmem_load_16x8(tmem + n + b * 8, v[b][0]);
                tmem_load_16x8(tmem + n + b * 8 + (16u << 16), v[b][1]);
            }
            tmem_wait(v[0]);
            tmem_wait(v[1]);
            const bool there = n + at < rows;
            const int64_t row = row0 + n + at;
            if (out != nullptr) {
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float(&s)[4] = v[i >> 1][i & 1];
                    p[i] = transpose_8x8(pack_bf16x2(activate(s[0], kept.act) * s[2], activate(s[1], kept.act) * s[3]));
                }
                const uint4 q = transpose_quad(p, c);
                if (there && f < F) st_v4(out + row * F + f, q);
            }
            if constexpr (KEEP != kNone) keep_block(v, row, there, f0, F, c);
        }
    }
};

// Few rows: a lane has one sum of G rows; the other projection's is eight lanes on.
template <Keep KEEP>
struct GatedFew : NoExtra {
    static constexpr bool kPairs = true, kStores = true;
    Kept kept;
    __device__ __forceinline__ void store(const float (&v)[kGroup], __nv_bfloat16* out, int64_t row0, int rows, int m, int M,
                                          int lane) const {
        const int side = lane >> 3 & 1, f = (m >> 4) * 8 + (m & 7), F = M / 2;
        const bool in = f < F;
#pragma unroll
        for (int j = 0; j < kGroup; j += 2) {
            if (j >= rows) break;
            // Lanes of Wg take row j, lanes of Wu row j + 1.
            const float other = __shfl_xor_sync(0xFFFFFFFFu, side ? v[j] : v[j + 1], 8);
            const float h = side ? activate(other, kept.act) * v[j + 1] : activate(v[j], kept.act) * other;
            if (out != nullptr && in && j + side < rows) store_half(out + (row0 + j + side) * F + f, h);
            if constexpr (KEEP == kBf16) {
                if (in) store_half(kept.halves(row0 + j, side) + f, v[j]);
                if (in && j + 1 < rows) store_half(kept.halves(row0 + j + 1, side) + f, v[j + 1]);
            } else if constexpr (KEEP == kE4m3) {
                // A group's 16 features are the lanes of one side.
                const uint32_t pair = pack_bf16x2(v[j], v[j + 1]);
                uint32_t most = larger_bf16x2(pair, pair);
#pragma unroll
                for (int i = 0; i < 4; ++i) most = larger_bf16x2(most, __shfl_xor_sync(0xFFFFFFFFu, most, i < 3 ? 1 << i : 16));
                const uint32_t e0 = kept_exponent(most & 0xFFFFu), e1 = kept_exponent(most >> 16);
                const uint32_t q = pack_e4m3x2(bf16_lo(pair) * kept_inverse(e0), bf16_hi(pair) * kept_inverse(e1));
                if (f < kept.padded) {
                    *(kept.bytes(row0 + j, side) + f) = (uint8_t)q;
                    if (j + 1 < rows) *(kept.bytes(row0 + j + 1, side) + f) = (uint8_t)(q >> 8);
                    if ((lane & 0x17) == 0) {
                        *kept.exponent(row0 + j, side, f) = (uint8_t)e0;
                        if (j + 1 < rows) *kept.exponent(row0 + j + 1, side, f) = (uint8_t)e1;
                    }
                }
            }
        }
    }
};

// ------------------------------------------------------------------ backward

struct Back {
    __nv_bfloat16* dgu;          // [rows][2][F]
    __nv_bfloat16* h;            // [rows][F], NULL to leave out
};

// The sums are dh. What was kept is read by rows, eight features a lane, and brought into the sums'
// layout by the transpositions of rows_of_features in reverse (its values are exact in bf16).
template <Keep KEEP>
struct GatedBackWide : NoExtra {
    Kept kept;
    Back to;
    // Eight features of one side, as four bf16 pairs.
    __device__ __forceinline__ uint4 load(int64_t row, int side, int f) const {
        if (KEEP == kBf16) return *reinterpret_cast<const uint4*>(kept.halves(row, side) + f);
        const uint2 q = *reinterpret_cast<const uint2*>(kept.bytes(row, side) + f);
        const float s = kept_scale(*kept.exponent(row, side, f));
        return make_uint4(kept_pair(q.x, s), kept_pair(q.x >> 16, s), kept_pair(q.y, s), kept_pair(q.y >> 16, s));
    }
    __device__ __forceinline__ void tile(uint32_t tmem, float*, unsigned char*, __nv_bfloat16*, int64_t row0, int rows, int m0,
                                         int M, int half, int lane) const {
        if (m0 >= M) return;
        const int g = lane >> 2, c = lane & 3, f = m0 + c * 8;
        for (int n = half * 8; n < rows; n += 16) {
            const bool there = n + g < rows && f < M;
            const int64_t row = row0 + n + g;
            uint32_t side[2][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (there) {
                    const uint4 q = load(row, h, f);
                    side[h][0] = q.x, side[h][1] = q.y, side[h][2] = q.z, side[h][3] = q.w;
                }
            float v[2][4];
            tmem_load_16x8(tmem + n, v[0]);
            tmem_load_16x8(tmem + n + (16u << 16), v[1]);
            tmem_wait(v);
            float dg[2][4], du[2][4], again[2][4];
            uint4 q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) q[h] = transpose_quad(side[h], c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t gate = transpose_8x8(i < 2 ? (i == 0 ? q[0].x : q[0].y) : (i == 2 ? q[0].z : q[0].w));
                const uint32_t up = transpose_8x8(i < 2 ? (i == 0 ? q[1].x : q[1].y) : (i == 2 ? q[1].z : q[1].w));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float u = j ? bf16_hi(up) : bf16_lo(up), dh = v[i >> 1][(i & 1) * 2 + j];
                    const Activated a = activate_both(j ? bf16_hi(gate) : bf16_lo(gate), kept.act);
                    dg[i >> 1][(i & 1) * 2 + j] = dh * u * a.slope;
                    du[i >> 1][(i & 1) * 2 + j] = dh * a.value;
                    again[i >> 1][(i & 1) * 2 + j] = a.value * u;
                }
            }
            const uint4 pg = rows_of_features(dg, c), pu = rows_of_features(du, c);
            if (there) {
                st_v4(to.dgu + 2 * row * M + f, pg);
                st_v4(to.dgu + (2 * row + 1) * M + f, pu);
            }
            if (to.h != nullptr) {
                const uint4 ph = rows_of_features(again, c);
                if (there) st_v4(to.h + row * M + f, ph);
            }
        }
    }
};

template <Keep KEEP>
struct GatedBackFew : NoExtra {
    static constexpr bool kStores = true;
    static constexpr int kGroup = 8;          // their loads are in flight together
    Kept kept;
    Back to;
    __device__ __forceinline__ float load(int64_t row, int side, int f) const {
        if (KEEP == kBf16) return __bfloat162float(*(kept.halves(row, side) + f));
        return kept_values(*(kept.bytes(row, side) + f)).x * kept_scale(*kept.exponent(row, side, f));
    }
    __device__ __forceinline__ void apply(float*, float (&)[kGroup], int64_t, int, int, int, int) const {}
    __device__ __forceinline__ void store(const float (&v)[kGroup], __nv_bfloat16*, int64_t row0, int rows, int m, int M, int) const {
        if (m >= M) return;
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            if (j >= rows) break;
            const int64_t row = row0 + j;
            const float u = load(row, 1, m);
            const Activated a = activate_both(load(row, 0, m), kept.act);
            store_half(to.dgu + 2 * row * M + m, v[j] * u * a.slope);
            store_half(to.dgu + (2 * row + 1) * M + m, v[j] * a.value);
            if (to.h != nullptr) store_half(to.h + row * M + m, a.value * u);
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

Kept kept_of(const ep_checkpoint* c, int F, int act) {
    Kept k{nullptr, nullptr, F, kept_features(F), act};
    if (c != nullptr) k.values = c->values, k.scales = c->scales;
    return k;
}

template <Direction D, class Wide, class Few>
ep_status run_block(const GemmMaps& maps, const GemmArgs& a, const Wide& wide, const Few& few, cudaStream_t stream) {
    const cudaError_t e = launch_gemm<D>(maps, a, wide, few, stream);
    return e == cudaSuccess ? EP_OK : cuda_fail(e);
}

// The maps of the rows, in boxes of a.box and of twice that.
ep_status encode_rows(GemmMaps* maps, const GemmArgs& a, const void* rows) {
    const uint64_t d[2] = {(uint64_t)a.C, (uint64_t)a.num_rows};
    uint32_t box[2] = {64, (uint32_t)a.box};
    const ep_status st = encode_map(&maps->b, rows, 2, d, box);
    if (st != EP_OK) return st;
    box[1] *= 2;
    return encode_map(&maps->b2, rows, 2, d, box);
}

template <Keep KEEP>
ep_status forward(const GemmMaps& maps, const GemmArgs& a, const Kept& kept, cudaStream_t stream) {
    GatedWide<KEEP> wide;
    GatedFew<KEEP> few;
    wide.kept = few.kept = kept;
    return run_block<kForward>(maps, a, wide, few, stream);
}

template <Keep KEEP>
ep_status backward(const GemmMaps& maps, const GemmArgs& a, const Kept& kept, const Back& to, cudaStream_t stream) {
    GatedBackWide<KEEP> wide;
    GatedBackFew<KEEP> few;
    wide.kept = few.kept = kept;
    wide.to = few.to = to;
    return run_block<kDgrad>(maps, a, wide, few, stream);
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status ep_expert_gated(const ep_gemm_shape* sh, const void* x, const void* w, const int32_t* expert_prefix, int32_t activation,
                          void* h, const ep_checkpoint* keep, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_block(sh, x, w, expert_prefix, activation, launch);
    if (st != EP_OK) return st;
    const bool rows = sh->num_rows > 0;
    if (keep != nullptr && (st = check_checkpoint(keep, rows, true)) != EP_OK) return st;
    if ((rows && h == nullptr && keep == nullptr) || ((uintptr_t)h & 15) != 0) return EP_ERR_INVALID_ARG;
    const uint64_t K = (uint64_t)sh->in_features, F = (uint64_t)sh->out_features, E = (uint64_t)sh->num_experts;
    GemmArgs a{};
    a.prefix = expert_prefix;
    a.out = reinterpret_cast<__nv_bfloat16*>(h);
    a.num_rows = sh->num_rows;
    a.E = sh->num_experts;
    a.M = 2 * sh->out_features;
    a.N = a.C = sh->in_features;
    a.err = launch->error_flags;
    gemm_tiles(&a, false);
    GemmMaps maps{};
    if (rows) {
        const uint64_t d[5] = {K, 8, 2, F / 8, E}, strides[4] = {2 * K, 2 * F * K, 16 * K, 4 * F * K};
        const uint32_t box[5] = {64, 8, 2, 8, 1};
        if ((st = encode_map(&maps.a, w, 5, d, box, strides)) != EP_OK) return st;
        if ((st = encode_rows(&maps, a, x)) != EP_OK) return st;
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        const Kept kept = kept_of(keep, sh->out_features, activation);
        st = keep == nullptr              ? forward<kNone>(maps, a, kept, launch->stream)
             : keep->dtype == EP_BF16 ? forward<kBf16>(maps, a, kept, launch->stream)
                                          : forward<kE4m3>(maps, a, kept, launch->stream);
        if (st != EP_OK) return st;
    }
    return end_call(launch);
}

ep_status ep_expert_gated_dgrad(const ep_gemm_shape* sh, const void* dy, const void* w, const int32_t* expert_prefix,
                                int32_t activation, const ep_checkpoint* kept, void* dgu, void* h, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_block(sh, dy, w, expert_prefix, activation, launch);
    if (st != EP_OK) return st;
    const bool rows = sh->num_rows > 0;
    if ((st = check_checkpoint(kept, rows, true)) != EP_OK) return st;
    if ((rows && dgu == nullptr) || (((uintptr_t)dgu | (uintptr_t)h) & 15) != 0) return EP_ERR_INVALID_ARG;
    GemmArgs a{};
    a.prefix = expert_prefix;
    a.num_rows = sh->num_rows;
    a.E = sh->num_experts;
    a.M = a.N = sh->in_features;
    a.C = sh->out_features;
    a.err = launch->error_flags;
    gemm_tiles(&a, false);
    GemmMaps maps{};
    if (rows) {
        const uint64_t d[3] = {(uint64_t)sh->in_features, (uint64_t)sh->out_features, (uint64_t)sh->num_experts};
        const uint32_t box[3] = {64, 64, 1};
        if ((st = encode_map(&maps.a, w, 3, d, box)) != EP_OK) return st;
        if ((st = encode_rows(&maps, a, dy)) != EP_OK) return st;
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        const Kept k = kept_of(kept, sh->in_features, activation);
        const Back to{reinterpret_cast<__nv_bfloat16*>(dgu), reinterpret_cast<__nv_bfloat16*>(h)};
        st = kept->dtype == EP_BF16 ? backward<kBf16>(maps, a, k, to, launch->stream) : backward<kE4m3>(maps, a, k, to, launch->stream);
        if (st != EP_OK) return st;
    }
    return end_call(launch);
}

}  // extern "C"
