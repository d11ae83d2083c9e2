// gemm.cuh -- the tensor-core product behind the experts' products and the adapters' projection.
#pragma once

#include <cuda.h>

#include <atomic>

#include "ep_internal.cuh"

namespace ep {

enum Direction { kForward, kDgrad, kWgrad };

struct GemmArgs {
    const int32_t* prefix;     // [E + 1]; NULL: one group of all rows
    __nv_bfloat16* out;
    int num_rows, E;
    int M;                     // forward: out_features, dgrad: in_features, wgrad: out_features
    int N;                     // wgrad: in_features (forward / dgrad: the rows)
    int C;                     // contracted features (wgrad: the rows)
    int bn, box, stages;       // columns of the widest tile, rows of one load box of B, stages
    int split;                 // CTAs that share a tile's contraction
    int smem;                  // bytes of dynamic shared memory
    int beside;                // of them beside the stages, for gemm_kernel's epilogue
    int loads = 0x7FFFFFFF;    // contracted values of a tile that are loaded: all, but in the self-test
    uint64_t wait_ns = 2000000000ull;      // bound on one barrier wait: 2 s, but in the self-test
    uint32_t* err;
};

struct GemmMaps {
    CUtensorMap a, b, b2, out;      // b2: b with boxes of twice the rows; out: wgrad's
    CUtensorMap other_b[2];         // b and b2 of the same rows in another order (Extra::reordered)
    CUtensorMap part_a[6], part_b[6];      // wgrad: a and b with boxes of 1, 2, 4, 8, 16, 32 rows
};

inline bool features_ok(int f) { return f >= 8 && f % 8 == 0; }
ep_status check_gemm_shape(const ep_gemm_shape* sh);

// Encodes a tiled bf16 map of up to five dimensions (innermost first), 128-byte swizzle. `strides`: bytes from
// one index of dimension i + 1 to the next; without them the dimensions follow one another.
ep_status encode_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint32_t* box,
                     const uint64_t* strides = nullptr);

// ------------------------------------------------------------------ expert rows

// Rows of expert e, clipped to the row buffers; end <= begin where there are none.
__device__ __forceinline__ int expert_begin(const GemmArgs& a, int e) {
    return a.prefix == nullptr ? 0 : min(max(a.prefix[e], 0), a.num_rows);
}
__device__ __forceinline__ int expert_end(const GemmArgs& a, int e) {
    return a.prefix == nullptr ? a.num_rows : min(max(a.prefix[e + 1], 0), a.num_rows);
}

// One warp: flags a prefix that leaves [0, num_rows] or decreases.
__device__ __forceinline__ void check_prefix(const GemmArgs& a, int lane) {
    if (a.prefix == nullptr) return;
    bool bad = false;
    for (int e = lane; e <= a.E; e += 32) {
        const int v = a.prefix[e];
        bad |= v < 0 || v > a.num_rows || (e < a.E && a.prefix[e + 1] < v);
    }
    if (bad) raise_flag(a.err, EP_DEVERR_RECV_OVERFLOW);
}

// ------------------------------------------------------------------ tensor memory, barriers

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Pair forms (cta_group::2): one thread of the leader CTA multiplies for both.
__device__ __forceinline__ void tmem_alloc2(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free2(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
// Arrives at the barrier at this offset in both CTAs.
__device__ __forceinline__ void tc_commit2(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tc_mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// 32 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_store_16x8(uint32_t at, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3])
                 : "memory");
}
// 8 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_store(uint32_t at, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 4, 8 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[4]) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 lanes (from the address's lane on) x 8 columns in the layout of a 16 x 8 product's sums: lane
// 4g + c has columns 2c, 2c+1 of lanes g (v[0], v[1]) and g + 8 (v[2], v[3]). The caller waits
// (tmem_wait) before it uses v.
__device__ __forceinline__ void tmem_load_16x8(uint32_t at, float (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_wait(float (&v)[2][4]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0][0]), "+f"(v[0][1]), "+f"(v[0][2]), "+f"(v[0][3]), "+f"(v[1][0]), "+f"(v[1][1]),
                   "+f"(v[1][2]), "+f"(v[1][3])::"memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_at(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Waits for a phase. Gives up when another role has (*dead), or after a.wait_ns (then flags
// EP_DEVERR_TIMEOUT and sets *dead): every role then leaves its loop. The global timer is first read
// after many tries.
static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* dead, uint32_t* err,
                                                   uint64_t wait_ns) {
    uint64_t t0 = 0;
    for (uint32_t n = 0;; ++n) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_at(bar, parity)) return true;
        if (*dead) return false;
        if ((n & 255) != 255) continue;
        if (t0 == 0) t0 = global_ns();
        if (global_ns() - t0 > wait_ns) {
            raise_flag(err, EP_DEVERR_TIMEOUT);
            *dead = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait_at(uint32_t bar, uint32_t parity, volatile int* dead, const GemmArgs& a) {
    if (mbar_try_at(bar, parity)) return true;
    return mbar_wait_slow(bar, parity, dead, a.err, a.wait_ns);
}
// `depth`: contracted values whose products are waited for too, each given kValueNs (a step of 64 takes a
// microsecond or less). 2^30 rows of one expert, 8 x 8 features: 3.9 s for the one tile of their wgrad.
constexpr uint64_t kValueNs = 64;
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* dead, const GemmArgs& a,
                                          int64_t depth = 0) {
    if (mbar_try_at(smem_addr(bar), parity)) return true;
    return mbar_wait_slow(smem_addr(bar), parity, dead, a.err, a.wait_ns + (depth > 0 ? (uint64_t)depth * kValueNs : 0));
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}

// Position in the ring of stages. The warps that issue loads and products must not take longer for a
// step than the step's product, so their loops hold no division by the number of stages (that
// alone kept the rate at 1.38 of 1.9 PFLOP/s), and the whole warp runs them, one elected lane
// issuing, so that addresses and descriptors stay in uniform registers.
struct Ring {
    uint32_t stages, s = 0, phase = 0;
    __device__ explicit Ring(uint32_t n) : stages(n) {}
    __device__ __forceinline__ void next() {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared-memory address in CTA `rank` of the cluster, and a value there.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    return at;
}
__device__ __forceinline__ float peer_value(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ int peer_word(uint32_t at) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void mbar_arrive_peer(uint32_t at) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}
__device__ __forceinline__ void mbar_expect_peer(uint32_t at, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(at), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_expect_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Pair loads: into this CTA's shared memory, completing on a barrier of either CTA (cluster address).
__device__ __forceinline__ void tma_load2_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load2_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load2_5d(uint32_t dst, const CUtensorMap* map, int x, int group, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %5, %5, %3, %4}], [%6];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(group), "r"(z), "r"(0), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// wgrad: the last `left` < 64 rows of an expert, 64 columns from x on. A product takes 16 rows at a time,
// and the rows that follow are another expert's, whose values may be infinite: so exactly the
// expert's rows are loaded, in boxes of powers of two, and the rest of the last 16 in boxes that lie beyond the tensor, which reads as zero. (Clearing them with stores and ordering
// those between the two CTAs cost a third of the whole product's time.)
template <bool PAIR>
__device__ __forceinline__ void load_tail_chunk(uint32_t at, const CUtensorMap* part, int x, int row, int left,
                                                int num_rows, uint32_t bar) {
    const int none = -left & 15;
    for (int bit = 5; bit >= 0; --bit)
        if (left >> bit & 1) {
            if (PAIR) tma_load2_2d(at, &part[bit], x, row, bar);
            else tma_load_2d_at(at, &part[bit], x, row, bar);
            at += 128 << bit;
            row += 1 << bit;
        }
    for (int bit = 3; bit >= 0; --bit)
        if (none >> bit & 1) {
            if (PAIR) tma_load2_2d(at, &part[bit], x, num_rows, bar);
            else tma_load_2d_at(at, &part[bit], x, num_rows, bar);
            at += 128 << bit;
        }
}

__device__ __forceinline__ void tma_load_3d_at(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d_at(uint32_t dst, const CUtensorMap* map, int x, int group, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %5, %5, %3, %4}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(group), "r"(z), "r"(0), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle (rows of 128 bytes, 8 rows a pattern).
//   K-major:  rows are M / N indices, 64 contracted values a row; 8-row groups 1024 bytes apart
//   MN-major: rows are contracted indices, 64 M / N values a row; 8-row groups 1024 bytes apart,
//             the next 64 M / N values kMnChunk bytes on
constexpr uint32_t kMnChunk = 64 * 128;
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn_major) {
    const uint64_t lbo = mn_major ? kMnChunk >> 4 : 1, sbo = 1024 >> 4;
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (lbo << 16) | (sbo << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32, M x n.
__device__ __forceinline__ uint32_t instr_desc(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ------------------------------------------------------------------ tiles

constexpr int kBM = 128, kBK = 64;
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr int kMaxStages = 8;
constexpr int kTileWarps = 8;          // writing warps of gemm_kernel, two per quarter of the lanes, but for extras with more

struct Tile {
    int e, m0, n0, n;          // expert, first M index, first column (row index or N index), columns
    int begin, end;            // the expert's rows
};

// Walks the tiles of all experts in order: expert by expert, in bands of four M tiles (of a pair's
// 256), column by column within a band: the tiles in work at a time then share their operands in
// L2 (8192^3: 662 -> 606 us; bands of 8 and 16: 647, 596; 32 experts of 512 rows: 350, 364, 366 us).
//   forward / dgrad: an expert's rows are cut into ceil(rows / bn) nearly even column tiles
//   wgrad:           N is cut into tiles of bn
// A tile's columns are a multiple of 32 (16 for each CTA).
constexpr int kBand = 4;
template <Direction D>
struct TileWalk {
    const GemmArgs& a;
    int e = -1, first = 0, count = 0, begin = 0, end = 0, mt, per = 0, nt = 0;
    __device__ TileWalk(const GemmArgs& args) : a(args), mt((args.M + 2 * kBM - 1) / (2 * kBM)) {}
    // Tile number t (non-decreasing from call to call); false past the last one.
    __device__ bool at(int t, Tile& out) {
        while (t >= first + count) {
            if (++e >= a.E) return false;
            first += count;
            begin = expert_begin(a, e);
            end = expert_end(a, e);
            const int rows = max(0, end - begin);
            if (D == kWgrad) {
                per = a.bn;
                nt = (a.N + a.bn - 1) / a.bn;
            } else {
                nt = (rows + a.bn - 1) / a.bn;
                per = nt > 0 ? ((rows + nt - 1) / nt + 31) & ~31 : 32;
                if (nt > 0) nt = (rows + per - 1) / per;
            }
            count = nt * mt;
        }
        const int q = t - first, band = q / (nt * kBand), width = min(kBand, mt - band * kBand);
        const int in = q - band * nt * kBand, c = in / width;
        out.e = e;
        out.m0 = (band * kBand + in - c * width) * 2 * kBM;
        out.begin = begin;
        out.end = end;
        if (D == kWgrad) {
            out.n0 = c * per;
            out.n = (min(per, a.N - out.n0) + 31) & ~31;
        } else {
            out.n0 = begin + c * per;
            out.n = (min(per, end - out.n0) + 31) & ~31;
        }
        return true;
    }
};

// Epilogue of G columns: forward / dgrad, few rows. A lane holds one feature of G rows; lanes exchange
// in pairs, so that a store covers 32 features of two rows (64 bytes each).
template <int G>
__device__ __forceinline__ void store_features(const float (&v)[G], __nv_bfloat16* out, int ld, int64_t row0, int rows,
                                               int feature, int M, int lane) {
#pragma unroll
    for (int j = 0; j < G; j += 2) {
        if (j >= rows) break;
        const bool odd = lane & 1;
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
        const uint32_t p = odd ? pack_bf16x2(other, v[j + 1]) : pack_bf16x2(v[j], other);
        const int jj = odd ? j + 1 : j;
        if (jj < rows && feature < M)
            *reinterpret_cast<uint32_t*>(out + (row0 + jj) * ld + (feature & ~1)) = p;
    }
}

// Transposes an 8 x 8 block of 16-bit values: lane 4g + c has columns 2c, 2c+1 of row g.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t t;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
    return t;
}
// Four 8 x 8 blocks of 16-bit values to and from shared memory, transposed: lane 4g + c has rows 2c, 2c+1 of
// column g of block i in word i; lane 8i + r gives the address of row r (16 bytes) of block i.
__device__ __forceinline__ void store_blocks(uint32_t at, const uint32_t (&v)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void load_blocks(uint32_t at, uint32_t (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Sums of 32 features x 8 rows in the layout of tmem_load_16x8 (lane 4g + c: rows 2c, 2c+1 of features
// g, 8 + g in v[0], 16 + g, 24 + g in v[1]) -> bf16, lane 4g + c the eight features 8c .. 8c+7 of row
// g: a transposition within 8 x 8 blocks and one within quads of lanes. A lane then stores 16
// bytes, a warp 64 bytes of eight rows.
__device__ __forceinline__ uint4 rows_of_features(const float (&v)[2][4], int c) {
    uint32_t p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        p[2 * t] = transpose_8x8(pack_bf16x2(v[t][0], v[t][1]));
        p[2 * t + 1] = transpose_8x8(pack_bf16x2(v[t][2], v[t][3]));
    }
#pragma unroll
    for (int bit = 1; bit <= 2; bit *= 2)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            if (h & bit) continue;
            const bool up = c & bit;
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? p[h] : p[h | bit], bit);
            if (up) p[h] = got;
            else p[h | bit] = got;
        }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// wgrad: a lane holds 64 consecutive columns of one row of dW; a warp stages its 32 rows x 64 columns
// in shared memory (16-byte pieces swizzled within 128-byte rows) and stores them with one bulk
// tensor copy, which leaves out what lies beyond dW's edges.
constexpr uint32_t kOutBytes = 32 * 128;
__device__ __forceinline__ void stage_columns(const float (&v)[32], uint32_t buf, int lane, int piece0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t at = buf + lane * 128 + (((piece0 + j) ^ (lane & 7)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack_bf16x2(v[8 * j], v[8 * j + 1])),
                     "r"(pack_bf16x2(v[8 * j + 2], v[8 * j + 3])), "r"(pack_bf16x2(v[8 * j + 4], v[8 * j + 5])),
                     "r"(pack_bf16x2(v[8 * j + 6], v[8 * j + 7]))
                     : "memory");
    }
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// What an epilogue adds to the sums before they are rounded; all writing threads make the calls together,
// each for output feature m. `shared`: kFloats floats of the block (gemm_split_kernel: kFewFloats).
// kFollows: the kernel directly follows one of this library after which the call's inputs are
// complete; only the epilogue waits for that kernel itself.
//   gemm_kernel:        tile writes rows row0 .. row0 + rows - 1 of a tile, features m0 .. m0 + 31, out of
//                       tensor memory; kWarps / 4 warps do, `half` 0, 1 and on. reordered: the rows are loaded
//                       through other_b. prepare is called by all writing threads before, while
//                       the products run. Both get a.beside bytes of shared memory
//   gemm_split_kernel:  ahead for the CTA's rows while the products run (before that wait), then apply
//                       for each kGroup of them: v[j] belongs to row row0 + c + j. Two halves of 128
//                       threads take groups in turn. kWrites: what is written is not the sums alone:
//                       write does it from tensor memory, as tile, where joined sums have gone back to
//                       and prefetch is called before for the rows, while the products run
// kPairs (forward): the M side is two projections of out_features each, eight rows of one and eight of the
// other in turn (maps.a has five dimensions: in_features, 8, 2, out_features / 8, experts).
struct NoExtra {
    static constexpr bool kFollows = false, kWrites = false, kPairs = false;
    static constexpr int kFloats = 4, kFewFloats = 4, kGroup = 32, kWarps = kTileWarps;
    __device__ __forceinline__ bool reordered() const { return false; }
    __device__ __forceinline__ void prepare(float*, unsigned char*, int64_t, int, int) const {}
    // Sixteen rows at a time, to have two blocks' steps in flight.
    __device__ __forceinline__ void tile(uint32_t tmem, float*, unsigned char*, __nv_bfloat16* out, int64_t row0, int rows,
                                         int m0, int M, int half, int lane) const {
        const int g = lane >> 2, c = lane & 3;
        const bool in = m0 + c * 8 < M;
        __nv_bfloat16* at = out + (row0 + g) * M + m0 + c * 8;
        for (int n = half * 16; n < rows; n += 32) {
            float v[2][2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tmem_load_16x8(tmem + n + b * 8, v[b][0]);
                tmem_load_16x8(tmem + n + b * 8 + (16u << 16), v[b][1]);
            }
            tmem_wait(v[0]);
            tmem_wait(v[1]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint4 p = rows_of_features(v[b], c);
                if (in && n + b * 8 + g < rows) st_v4(at + (int64_t)(n + b * 8) * M, p);
            }
        }
    }
    __device__ __forceinline__ void ahead(float*, int64_t, int, int, int) const {}
    __device__ __forceinline__ void apply(float*, float (&)[32], int64_t, int, int, int, int) const {}
};

// The epilogue's THREADS: a barrier, and whether all of them have `mine` (the same answer to all, so
// that none waits at a later barrier that another has left out).
template <int THREADS>
__device__ __forceinline__ void epilogue_barrier(int id = 1) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ bool epilogue_all(bool mine) {
    uint32_t all;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.and.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(all)
        : "r"((uint32_t)mine), "n"(THREADS)
        : "memory");
    return all != 0;
}

// D[m][n] over tiles of 256 x up to 256, a pair of CTAs per tile (cta_group::2), each pair walking over
// tiles. The weights are the M side and the rows the N side, so that a tile has as many columns as
// its expert has rows left (to a multiple of 32): no padding of the experts. Each CTA loads its 128 of
// the M side and half of the columns; the tensor cores of both read both halves, which halves the
// shared memory traffic of the columns. Warp 0 loads the M side (TMA), warp 1 of the leader
// multiplies (tcgen05.mma, fp32 sums in tensor memory, two accumulators of 256 columns in turn),
// warp 3 loads the columns, warps 4 on write the tile before meanwhile; wgrad: warp 2 loads the
// tails. Full tiles are bound by the tensor cores (8192^3 1.90 PFLOP/s; 32771 rows of 32 experts,
// 7168 -> 4096: 1.27 ms, tensor pipe 91 % active), narrower ones by filling shared memory (512 rows
// an expert, 7168 -> 2048: dgrad 79 %, wgrad with its 8 steps a tile 62 %).
//   full[s]   leader's: both CTAs' loads (an arrival of each loading warp, and the bytes)
//   empty[s]  each CTA's: the products that read stage s are done
template <Direction D, class Extra>
__global__ void __launch_bounds__(128 + 32 * Extra::kWarps, 1)
    gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs a, const Extra extra) {
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int dead;
    __shared__ __align__(16) float s_extra[Extra::kFloats];
    constexpr bool kAMn = D != kForward, kBMn = D == kWgrad;
    unsigned char* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t stage_bytes = kABytes + (uint32_t)a.bn * 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.x / 2, step = gridDim.x / 2;
    // wgrad keeps its last stage for the tails, whose many small boxes a warp of its own issues: they take
    // longer than the ring is ahead (32 experts of 511 rows, 7168 x 2048: 397 -> 334 us).
    const uint32_t ring_stages = D == kWgrad ? a.stages - 1 : a.stages;

    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&maps.a);
        tma_prefetch_map(&maps.b);
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], D == kWgrad && s == a.stages - 1 ? 2 : 4);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * Extra::kWarps);
        }
        mbar_init(&drain, 1);
        dead = 0;
    }
    __syncwarp();
    if (warp == 1) tmem_alloc2(&s_tmem, 512);
    tc_fence_before();
    __syncwarp();
    cluster_barrier();          // the barriers and the tensor memory of both CTAs are there
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (!Extra::kFollows || warp >= 4) pdl_wait();

    if (warp == 0 || warp == 3) {
        // Warp 0 loads the M side, warp 3 the columns.
        if (warp == 3 && blockIdx.x == 0) check_prefix(a, lane);
        TileWalk<D> walk(a);
        Tile t;
        Ring ring(ring_stages);
        bool ok = true;
        const uint32_t full0 = peer_addr(smem_addr(full), 0);
        const uint32_t empty0 = smem_addr(empty), smem0 = smem_addr(smem) + (warp == 0 ? 0 : kABytes);
        const bool reordered = extra.reordered();
        const CUtensorMap* map = warp == 0 ? &maps.a : reordered ? &maps.other_b[0] : &maps.b;
        const CUtensorMap* map2 = reordered ? &maps.other_b[1] : &maps.b2;
        for (int i = first; ok && walk.at(i, t); i += step) {
            const int depth = D == kWgrad ? t.end - t.begin : a.C;
            const int half = t.n / 2, m0 = t.m0 + (int)rank * kBM, n0 = t.n0 + (int)rank * half;
            const int box = kBMn ? 64 : half > 64 ? 2 * a.box : a.box, boxes = (half + box - 1) / box;
            const uint32_t bytes = warp == 0 ? kABytes : (uint32_t)(boxes * box) * 128;
            const int whole = D == kWgrad ? depth & ~(kBK - 1) : depth, upto = min(whole, a.loads);
            for (int k0 = 0; k0 < upto; k0 += kBK, ring.next()) {
                if (!(ok = mbar_wait_at(empty0 + ring.s * 8, ring.phase ^ 1, &dead, a))) break;
                const uint32_t at = smem0 + ring.s * stage_bytes, bar = full0 + ring.s * 8;
                if (elect_one()) {
                    mbar_expect_peer(bar, bytes);
                    if (warp == 0) {
                        if constexpr (Extra::kPairs) {
                            tma_load2_5d(at, map, k0, m0 / 16, t.e, bar);
                        } else if (D == kForward) {
                            tma_load2_3d(at, map, k0, m0, t.e, bar);
                        } else if (D == kDgrad) {
                            tma_load2_3d(at, map, m0, k0, t.e, bar);
                            tma_load2_3d(at + kMnChunk, map, m0 + 64, k0, t.e, bar);
                        } else {
                            tma_load2_2d(at, map, m0, t.begin + k0, bar);
                            tma_load2_2d(at + kMnChunk, map, m0 + 64, t.begin + k0, bar);
                        }
                    } else if (kBMn) {
                        for (int b = 0; b < boxes; ++b) tma_load2_2d(at + b * kMnChunk, map, n0 + b * 64, t.begin + k0, bar);
                    } else {
                        tma_load2_2d(at, half > 64 ? map2 : map, k0, n0, bar);
                    }
                }
                __syncwarp();
            }
            ok = ok && upto == whole;
        }
        // The last loads' stages are free: nothing more arrives at this CTA's barriers. (Where a role has
        // given up, that is waited for as long as copies in flight may take.)
        if (warp == 0) {
            for (uint32_t q = 0; q < ring_stages; ++q, ring.next())
                ok = mbar_wait_bounded(&empty[ring.s], ring.phase ^ 1, ok ? a.wait_ns : a.wait_ns / 64) && ok;
        }
    } else if (D == kWgrad && warp == 2) {
        // The tails, into their own stage as soon as the tile before has been multiplied.
        TileWalk<D> walk(a);
        Tile t;
        uint32_t tails = 0;
        int64_t rows = 0, pending = 0;          // of the tiles since the last tail's, and up to that one's
        bool ok = true;
        const uint32_t bar = peer_addr(smem_addr(&full[ring_stages]), 0), at = smem_addr(smem) + ring_stages * stage_bytes;
        for (int i = first; ok && walk.at(i, t); i += step) {
            const int depth = t.end - t.begin, left = depth > 0 ? depth % kBK : 0;
            rows += max(depth, 0);
            if (left == 0) continue;
            if (!(ok = depth <= a.loads)) break;
            if (!(ok = mbar_wait(&empty[ring_stages], (tails & 1) ^ 1, &dead, a, pending))) break;
            pending = rows;
            rows = 0;
            ++tails;
            if (elect_one()) {
                const int half = t.n / 2, boxes = (half + 63) / 64;
                mbar_expect_peer(bar, (uint32_t)((2 + boxes) * ((left + 15) & ~15)) * 128);
                for (int c = 0; c < 2 + boxes; ++c)
                    load_tail_chunk<true>(at + c * kMnChunk, c < 2 ? maps.part_a : maps.part_b,
                                          c < 2 ? t.m0 + (int)rank * kBM + c * 64 : t.n0 + (int)rank * half + (c - 2) * 64,
                                          t.end - left, left, a.num_rows, bar);
            }
            __syncwarp();
        }
        mbar_wait_bounded(&empty[ring_stages], (tails & 1) ^ 1, ok ? a.wait_ns : a.wait_ns / 64);
    } else if (warp == 1 && rank == 0) {
        TileWalk<D> walk(a);
        Tile t;
        Ring ring(ring_stages);
        uint32_t used = 0, tails = 0;
        bool ok = true;
        const uint32_t full0 = smem_addr(full), empty0 = smem_addr(empty);
        const uint64_t da0 = smem_desc(smem_addr(smem), kAMn), db0 = smem_desc(smem_addr(smem) + kABytes, kBMn);
        for (int i = first; ok && walk.at(i, t); i += step) {
            const int depth = D == kWgrad ? t.end - t.begin : a.C;
            if (depth <= 0) continue;
            const uint32_t acc = used & 1;
            if (!(ok = mbar_wait(&acc_empty[acc], ((used >> 1) & 1) ^ 1, &dead, a))) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * 256, idesc = instr_desc(2 * kBM, t.n, kAMn, kBMn);
            for (int k0 = 0; k0 < depth; k0 += kBK) {
                const int left = depth - k0;
                uint32_t s = ring.s, phase = ring.phase;
                if (D == kWgrad && left < kBK) s = ring_stages, phase = tails++ & 1;
                else ring.next();
                if (!(ok = mbar_wait_at(full0 + s * 8, phase, &dead, a))) break;
                tc_fence_after();
                const uint64_t at = (uint64_t)((s * stage_bytes) >> 4), da = da0 + at, db = db0 + at;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBK; k += 16) {
                        if (k >= left) break;      // 16 contracted values: 32 bytes of a row, or 16 rows
                        tc_mma2(d, da + (kAMn ? k * 128 : k * 2) / 16, db + (kBMn ? k * 128 : k * 2) / 16, idesc, (k0 | k) != 0);
                    }
                    tc_commit2(empty0 + s * 8);
                }
                __syncwarp();
            }
            if (!ok) break;          // the tile is not complete: neither CTA may write it
            if (elect_one()) tc_commit2(smem_addr(&acc_full[acc]));
            __syncwarp();
            ++used;
        }
        if (!ok) {
            if (elect_one()) tc_commit2(smem_addr(&drain));
            __syncwarp();
            mbar_wait_bounded(&drain, 0, a.wait_ns / 8);
        }
    } else if (warp >= 4) {
        TileWalk<D> walk(a);
        Tile t;
        uint32_t used = 0;
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t out0 = smem_addr(smem) + a.stages * stage_bytes + (warp - 4) * kOutBytes;     // wgrad
        for (int i = first; walk.at(i, t); i += step) {
            const bool some = D != kWgrad || t.end > t.begin;
            const uint32_t acc = used & 1;
            const int rows = min(t.n, t.end - t.n0);
            if (D != kWgrad) extra.prepare(s_extra, smem + a.stages * stage_bytes, t.n0, rows, t.m0 + (int)rank * kBM);
            if (some) {
                const bool there = mbar_wait(&acc_full[acc], (used >> 1) & 1, &dead, a, D == kWgrad ? t.end - t.begin : a.C);
                if (!epilogue_all<32 * Extra::kWarps>(there)) break;
                tc_fence_after();
            }
            const int m = t.m0 + (int)rank * kBM + quarter * 32 + lane;
            if constexpr (D == kWgrad) {
                const int m_warp = t.m0 + (int)rank * kBM + quarter * 32;
                for (int c = half * 64; m_warp < a.M && c < t.n; c += 128) {
                    const uint32_t buf = out0;
                    if (lane == 0) bulk_wait_smem_read();      // this buffer's last store has read it
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[32];
                        if (some) {
                            tmem_load(tmem + acc * 256 + c + h * 32 + ((uint32_t)quarter << 21), v);
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                        }
                        stage_columns(v, buf, lane, h * 4);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&maps.out, buf, t.n0 + c, m_warp, t.e);
                        bulk_commit();
                    }
                }
            } else {
                extra.tile(tmem + acc * 256 + ((uint32_t)quarter << 21), s_extra, smem + a.stages * stage_bytes, a.out, t.n0, rows,
                           m - lane, a.M, half, lane);
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_peer(peer_addr(smem_addr(&acc_empty[acc]), 0));
                ++used;
            }
        }
        if (D == kWgrad && lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    cluster_barrier();          // both are done with each other's barriers and tensor memory
    if (warp == 1) tmem_free2(tmem, 512);
    pdl_trigger();
}

// ------------------------------------------------------------------ few rows: split contraction

// One warp: tile number i of all experts, M tiles of 128 innermost; forward / dgrad: 32 experts at a time;
// false past the last one.
template <Direction D>
__device__ __forceinline__ bool find_tile(const GemmArgs& a, int i, int lane, Tile& out) {
    const int mt = (a.M + kBM - 1) / kBM;
    if (D == kWgrad) {
        const int nt = (a.N + a.bn - 1) / a.bn, e = i / (mt * nt), c = i / mt % nt;
        if (e >= a.E) return false;
        out.e = e;
        out.m0 = i % mt * kBM;
        out.n0 = c * a.bn;
        out.n = (min(a.bn, a.N - out.n0) + 15) & ~15;
        out.begin = expert_begin(a, e);
        out.end = max(out.begin, expert_end(a, e));
        return true;
    }
    int first = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        int begin = 0, end = 0;
        if (e < a.E) {
            begin = expert_begin(a, e);
            end = expert_end(a, e);
        }
        const int rows = max(0, end - begin), cut = (rows + a.bn - 1) / a.bn;
        const int per = cut > 0 ? ((rows + cut - 1) / cut + 15) & ~15 : 16;
        const int count = (rows + per - 1) / per * mt;
        int upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += up;
        }
        const int start = first + upto - count;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, i >= start && i < start + count);
        if (hit != 0) {
            const int src = __ffs(hit) - 1, q = i - start, c = q / mt;
            Tile t{e, (q - c * mt) * kBM, begin + c * per, 0, begin, end};
            t.n = (min(per, end - t.n0) + 15) & ~15;
            out.e = __shfl_sync(0xFFFFFFFFu, t.e, src);
            out.m0 = __shfl_sync(0xFFFFFFFFu, t.m0, src);
            out.n0 = __shfl_sync(0xFFFFFFFFu, t.n0, src);
            out.n = __shfl_sync(0xFFFFFFFFu, t.n, src);
            out.begin = __shfl_sync(0xFFFFFFFFu, t.begin, src);
            out.end = __shfl_sync(0xFFFFFFFFu, t.end, src);
            return true;
        }
        first += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    return false;
}

constexpr int kSplitThreads = 320;

// The writing warps of a CTA that has given up: NaN for its whole part, once copies in flight have had
// time to land (they share the memory).
static __device__ __noinline__ void spoil_part(float* part, int columns, uint64_t* done, uint64_t wait_ns) {
    mbar_wait_bounded(done, 0, wait_ns);
    for (int i = threadIdx.x - 64; i < columns * kBM; i += kSplitThreads - 64) part[i] = __int_as_float(0x7FFFFFFF);
}
// Whether all parts of the tile are complete (`complete`: this CTA's word of that).
static __device__ __noinline__ bool parts_complete(const int* complete, int split) {
    bool all = true;
    for (int r = 0; r < split; ++r) all = all && peer_word(peer_addr(smem_addr(complete), r)) != 0;
    return all;
}

// Where rows are few and the weights are what is read (forward, dgrad), or where tiles are few and the
// rows many (wgrad): a cluster of `split` CTAs per tile, each over its part of the contraction, so
// that enough CTAs stream weights at the same time (and two fit an SM, one filling its pipeline
// while the other runs). Each CTA leaves its fp32 part in its own shared memory; after a cluster
// barrier each adds up, in rank order, the parts of its share of the rows. Warp 0 loads, warp 1
// multiplies, warps 2 to 9 write. Bound by the stream of weights (251 rows of 32 experts, 7168 ->
// 2048: 136 us, 6.9 TB/s), a single small matrix by launch, pipeline fill and the join (one row 7168
// x 7168: 21 us, 4096 x 4096: 10).
template <Direction D, class Extra>
__global__ void __launch_bounds__(kSplitThreads, 2)
    gemm_split_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs a, const Extra extra) {
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], done, drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int dead;
    __shared__ __align__(16) float s_extra[Extra::kFewFloats];
    __shared__ Tile s_tile;
    __shared__ int s_has;
    __shared__ int s_complete;             // this CTA's part is
    constexpr bool kAMn = D != kForward, kBMn = D == kWgrad;
    unsigned char* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t stage_bytes = kABytes + (uint32_t)a.bn * 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.split > 1 ? (int)cluster_rank() : 0;

    if (threadIdx.x == 0) {
        tma_prefetch_map(&maps.a);
        tma_prefetch_map(&maps.b);
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        mbar_init(&drain, 1);
        dead = 0;
    }
    if (warp == 1) tmem_alloc(&s_tmem, (uint32_t)a.bn);
    if (!Extra::kFollows) pdl_wait();
    if (warp == 2) {
        Tile t{};
        const bool has = find_tile<D>(a, blockIdx.x / a.split, lane, t);
        if (lane == 0) {
            s_tile = t;
            s_has = has;
        }
    }
    if (warp == 3 && blockIdx.x == 0) check_prefix(a, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Tile t = s_tile;
    const bool has = s_has;            // the same in all CTAs of a cluster
    const int depth = D == kWgrad ? t.end - t.begin : a.C, blocks = (depth + kBK - 1) / kBK;
    const int kb0 = (int)((int64_t)blocks * rank / a.split), kb1 = (int)((int64_t)blocks * (rank + 1) / a.split);

    if (has && warp == 0) {
        const int boxes = (t.n + a.box - 1) / a.box;
        const uint32_t bytes = kABytes + (uint32_t)boxes * a.box * 128, smem0 = smem_addr(smem);
        const uint32_t full0 = smem_addr(full), empty0 = smem_addr(empty);
        Ring ring(a.stages);
        bool ok = true;
        const int upto = min(kb1, a.loads / kBK);
        for (int kb = kb0; kb < upto; ++kb, ring.next()) {
            if (!(ok = mbar_wait_at(empty0 + ring.s * 8, ring.phase ^ 1, &dead, a))) break;
            const uint32_t sa = smem0 + ring.s * stage_bytes, sb = sa + kABytes, bar = full0 + ring.s * 8;
            const int k0 = kb * kBK, left = depth - k0;
            if (elect_one()) {
                if (D == kWgrad && left < kBK && (left & 15) != 0) {
                    mbar_expect_at(bar, (uint32_t)((2 + boxes) * ((left + 15) & ~15)) * 128);
                    for (int c = 0; c < 2 + boxes; ++c)
                        load_tail_chunk<false>(sa + c * kMnChunk, c < 2 ? maps.part_a : maps.part_b,
                                               c < 2 ? t.m0 + c * 64 : t.n0 + (c - 2) * 64, t.begin + k0, left, a.num_rows, bar);
                } else {
                    mbar_expect_at(bar, bytes);
                    if (Extra::kPairs) {
                        tma_load_5d_at(sa, &maps.a, k0, t.m0 / 16, t.e, bar);
                    } else if (D == kForward) {
                        tma_load_3d_at(sa, &maps.a, k0, t.m0, t.e, bar);
                    } else if (D == kDgrad) {
                        tma_load_3d_at(sa, &maps.a, t.m0, k0, t.e, bar);
                        tma_load_3d_at(sa + kMnChunk, &maps.a, t.m0 + 64, k0, t.e, bar);
                    } else {
                        tma_load_2d_at(sa, &maps.a, t.m0, t.begin + k0, bar);
                        tma_load_2d_at(sa + kMnChunk, &maps.a, t.m0 + 64, t.begin + k0, bar);
                    }
                    for (int b = 0; b < boxes; ++b) {
                        if (kBMn) tma_load_2d_at(sb + b * kMnChunk, &maps.b, t.n0 + b * 64, t.begin + k0, bar);
                        else tma_load_2d_at(sb + b * a.box * 128, &maps.b, k0, t.n0 + b * a.box, bar);
                    }
                }
            }
            __syncwarp();
        }
        if (!ok || upto < kb1)     // wait, with a limit, for the copies still in flight
            for (int s = 0; s < a.stages; ++s, ring.next()) mbar_wait_bounded(&empty[ring.s], ring.phase ^ 1, a.wait_ns / 64);
    } else if (has && warp == 1) {
        const uint32_t idesc = instr_desc(kBM, t.n, kAMn, kBMn), full0 = smem_addr(full), empty0 = smem_addr(empty);
        const uint64_t da0 = smem_desc(smem_addr(smem), kAMn), db0 = smem_desc(smem_addr(smem) + kABytes, kBMn);
        Ring ring(a.stages);
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
            if (!(ok = mbar_wait_at(full0 + ring.s * 8, ring.phase, &dead, a))) break;
            tc_fence_after();
            const uint64_t at = (uint64_t)((ring.s * stage_bytes) >> 4), da = da0 + at, db = db0 + at;
            const int left = depth - kb * kBK;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBK; k += 16) {
                    if (D == kWgrad && k >= left) break;
                    tc_mma(tmem, da + (kAMn ? k * 128 : k * 2) / 16, db + (kBMn ? k * 128 : k * 2) / 16, idesc, kb > kb0 || k > 0);
                }
                tc_commit(empty0 + ring.s * 8);
            }
            __syncwarp();
        }
        if (elect_one()) tc_commit(smem_addr(ok ? &done : &drain));      // done: this part is complete
        __syncwarp();
        if (!ok) mbar_wait_bounded(&drain, 0, a.wait_ns / 8);
    }
    __syncwarp();
    const int quarter = warp & 3, half = (warp - 2) >> 2, m_local = quarter * 32 + lane, m = t.m0 + m_local;
    // Columns of the tile (rows; wgrad: in_features, eight at a time), and this CTA's share of them.
    const int rows = D == kWgrad ? min(t.n, a.N - t.n0) : min(t.n, t.end - t.n0), unit = D == kWgrad ? 8 : 1;
    const int share = (rows + a.split * unit - 1) / (a.split * unit) * unit, lo = rank * share, hi = min(rows, lo + share);
    bool ok = has;
    if (has && warp >= 2) {
        if constexpr (Extra::kWrites) extra.prefetch(t.n0 + lo, hi - lo, t.m0, threadIdx.x - 64, 256);
        if (D != kWgrad) extra.ahead(s_extra, t.n0 + lo, hi - lo, m, half);
        ok = epilogue_all<256>(mbar_wait(&done, 0, &dead, a, (kb1 - kb0) * kBK));
        tc_fence_after();
    }
    if (Extra::kFollows && warp >= 2) pdl_wait();
    constexpr int G = Extra::kGroup;
    const bool some = kb1 > kb0;
    if (D != kWgrad && a.split == 1) {
        if constexpr (Extra::kWrites) {
            if (ok && warp >= 2)
                extra.template write<2>(tmem + ((uint32_t)quarter << 21), smem_addr(s_extra), a.out, t.n0, rows,
                                        m - lane, a.M, half, lane);
        } else if (ok && warp >= 2) {
            for (int c = half * G; c < rows; c += 2 * G) {
                float v[G];
                tmem_load(tmem + c + ((uint32_t)quarter << 21), v);
                extra.apply(s_extra, v, t.n0, rows, c, m, half);
                store_features(v, a.out, a.M, t.n0 + c, rows - c, m, a.M, lane);
            }
        }
    } else {
        float* part = reinterpret_cast<float*>(smem);      // [columns][128]; every product has read its stage
        if (ok && warp >= 2) {
            for (int c = half * 8; c < rows; c += 16) {
                float v[8];
                if (some) {
                    tmem_load(tmem + c + ((uint32_t)quarter << 21), v);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) part[(c + j) * kBM + m_local] = v[j];     // up to bn columns
            }
        }
        // The tile is written where every part is complete. A CTA that has given up leaves NaN as its part,
        // so that the others ask for its word only then: asking every time, before or beside the sums,
        // took 0.2 to 0.4 us of the 10 that one row 4096 x 4096 takes.
        if (threadIdx.x == 64) s_complete = ok;          // (warp 2's ok is that of all writing warps)
        if (has && !ok && warp >= 2) spoil_part(part, a.bn, &done, a.wait_ns / 64);
        __syncwarp();
        cluster_barrier();
        const uint32_t at = smem_addr(part);
        if constexpr (D == kWgrad) {
            for (int c = lo + half * 8; ok && warp >= 2 && m < a.M && c < hi; c += 16) {
                float v[8] = {};
                for (int r = 0; r < a.split; ++r) {
                    const uint32_t peer = peer_addr(at, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += peer_value(peer + ((c + j) * kBM + m_local) * 4);
                }
                if (isnan(v[0]) && !parts_complete(&s_complete, a.split)) break;
                st_v4(a.out + ((int64_t)t.e * a.M + m) * a.N + t.n0 + c,
                      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
            }
        } else if constexpr (Extra::kWrites) {
            // The joined sums go back to tensor memory, from its first column on.
            bool fine = ok;
            for (int c = lo + half * 8; ok && warp >= 2 && c < hi; c += 16) {
                float v[8] = {};
                for (int r = 0; r < a.split; ++r) {
                    const uint32_t peer = peer_addr(at, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < hi) v[j] += peer_value(peer + ((c + j) * kBM + m_local) * 4);
                }
                fine = fine && (!isnan(v[0]) || parts_complete(&s_complete, a.split));
                tmem_store(tmem + c - lo + ((uint32_t)quarter << 21), v);
            }
            if (warp >= 2) {
                tmem_store_wait();
                tc_fence_before();
                fine = epilogue_all<256>(fine);
                tc_fence_after();
                if (fine)
                    extra.template write<2>(tmem + ((uint32_t)quarter << 21), smem_addr(s_extra), a.out,
                                            t.n0 + lo, hi - lo, m - lane, a.M, half, lane);
            }
        } else if (ok && warp >= 2 && lo < hi) {
            for (int c = lo + half * G; c < hi; c += 2 * G) {
                float v[G];
#pragma unroll
                for (int j = 0; j < G; ++j) v[j] = 0.0f;
                for (int r = 0; r < a.split; ++r) {
                    const uint32_t peer = peer_addr(at, r);
#pragma unroll
                    for (int j = 0; j < G; ++j)
                        if (c + j < hi) v[j] += peer_value(peer + ((c + j) * kBM + m_local) * 4);
                }
                const bool failed = isnan(v[0]) && !parts_complete(&s_complete, a.split);          // for all alike
                extra.apply(s_extra, v, t.n0 + lo, hi - lo, c - lo, m, half);
                if (!__any_sync(0xFFFFFFFFu, failed)) store_features(v, a.out, a.M, t.n0 + c, hi - c, m, a.M, lane);
            }
        }
        __syncwarp();
        cluster_barrier();          // until here the peers read this CTA's shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free(tmem, (uint32_t)a.bn);
    pdl_trigger();
}

// ------------------------------------------------------------------ host

// How many tiles of `wide` M indices there can be at most: one for each expert's first row, one more for
// every bn rows.
inline int64_t gemm_most_tiles(const GemmArgs& a, bool wgrad, int wide) {
    const int64_t mt = ceil_div(a.M, wide), some = a.E < a.num_rows ? a.E : a.num_rows;
    return mt * (wgrad ? (int64_t)a.E * ceil_div(a.N, a.bn) : some + (a.num_rows - some) / a.bn);
}

// Whether gemm_split_kernel runs (else gemm_kernel). (In clusters of at least two also for wgrad.)
inline bool gemm_by_split(const GemmArgs& a) { return a.bn <= 64 || a.split > 1; }

// Column tile width, stages and split.
//   wgrad: tiles of 256 columns, a pair of CTAs each; where those are less than half of the pairs
//          and experts have many rows, tiles of 128 x 128 whose rows are split (one expert of 7568 rows,
//          672 -> 392 features: 40 -> 17 us).
//   else:  tiles of twice the average rows of an expert (one group: of its rows), within [32, widest],
//          so that most experts are one tile. Up to 64 columns the weights' loads are what counts:
//          two CTAs per SM, and the contraction split as long as all CTAs fit at once (one row,
//          7168 x 7168: 4 parts 21 us, 8 parts, more CTAs than fit, 35 us); wider tiles are split only
//          where there are fewer of them than SMs. Before it is split further, a part has sixteen
//          64-deep steps or more (wider tiles: 32; below, pairs of CTAs are as fast and write faster).
//   Adapters, whose work for the rows counts too, pass: the most rows of a wider tile that a part may
//          have; the fewest steps (`least`) with which CTAs for up to half of the SMs are split further (24
//          rows 512 -> 512, rank 64: 4 steps 11 us, 16 steps 17).
// Narrow tiles that are few take an SM each: 128 KB, so that two do not share one while others are
// idle (128 rows 1024 -> 4096 with adapters of rank 64, 128 CTAs: 23 us, else 31). Not in clusters of
// eight: an SM each, not all of them fit at once (70 rows 4096 -> 1024: 17 us, else 12).
inline void gemm_tiles(GemmArgs* a, bool wgrad, int beside = 0, int most_rows = 256, int widest = 256, int least = 16,
                       int most_parts = 8) {
    int bn = 256;
    const int avg = (a->num_rows + a->E - 1) / a->E, wide = a->E > 1 ? 2 * (avg < 256 ? avg : 256) : avg;
    if (!wgrad)
        for (bn = 32; bn < widest && bn < wide; bn *= 2) {}
    a->bn = bn;
    a->box = bn < 64 ? bn : 64;
    a->split = 1;
    const int sms = sm_count();
    if (!wgrad) {
        const int64_t tiles = (int64_t)ceil_div(a->M, kBM) * (a->E < a->num_rows ? a->E : a->num_rows) * ceil_div(avg, bn);
        const int64_t want = bn <= 64 ? 2 * sms : sms;
        const int steps = ceil_div(a->C, kBK);
        while (a->split < most_parts && tiles * a->split * 2 <= want &&
               steps >= a->split * (bn > 64 ? 32 : tiles * a->split * 2 <= sms / 2 ? least : 16))
            a->split *= 2;
        if (bn > 64 && (avg < bn ? avg : bn) > most_rows * a->split) a->split = 1;
    }
    if (wgrad && 2 * gemm_most_tiles(*a, true, 2 * kBM) <= sms / 2 && avg >= 16 * kBK) {
        a->bn = 128;
        const int64_t tiles = gemm_most_tiles(*a, true, kBM);
        while (a->split < 8 && tiles * a->split * 2 <= sms && avg >= a->split * 8 * kBK) a->split *= 2;
        if (a->split == 1) a->bn = 256;
    }
    bn = a->bn;
    const bool split = gemm_by_split(*a);
    const bool spread = a->split <= 4 && gemm_most_tiles(*a, wgrad, kBM) * a->split <= sms;
    const int stage = (int)kABytes + (split ? bn * 128 : bn * 64), room = (split && bn <= 64 ? spread ? 128 : 96 : 200) * 1024;
    a->beside = split ? 0 : wgrad ? 8 * (int)kOutBytes : beside;
    const int left = (wgrad ? 224 : 220) * 1024 - a->beside, most = split || left > room ? room : left;
    a->stages = most / stage < kMaxStages ? most / stage : kMaxStages;
    a->smem = a->stages * stage + 1024 + a->beside;
}

constexpr int kSplitSmemMax = 201 * 1024, kGemmSmemMax = 222 * 1024, kWgradSmemMax = 225 * 1024;

// WHICH: a number of its own for each kernel with this Extra. Its shared-memory limit is set once per device (0.6 us of
// a call's 4 on the host): the runtime holds it for all of the device's contexts, and for one that was reset.
template <int WHICH, class Kernel, class Extra>
cudaError_t launch_gemm_as(Kernel kernel, int smem_most, unsigned blocks, unsigned threads, unsigned cluster, cudaStream_t stream,
                           const GemmMaps& maps, const GemmArgs& a, const Extra& extra) {
    static std::atomic<uint64_t> set[2];
    const int beside = 227 * 1024 - 512 - Extra::kFloats * 4;          // what the kernel's own arrays leave
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device < 0 || device >= 128) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << (device & 63);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)a.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if ((set[device >> 6].load(std::memory_order_relaxed) & bit) == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_most < beside ? smem_most : beside);
        if (e != cudaSuccess) return e;
        set[device >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    e = cudaLaunchKernelEx(&cfg, kernel, maps, a, extra);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// Launches the product (a.num_rows > 0) as gemm_tiles has laid it out.
template <Direction D, class Wide, class Few>
cudaError_t launch_gemm(const GemmMaps& maps, const GemmArgs& a, const Wide& wide, const Few& few, cudaStream_t stream) {
    if (gemm_by_split(a)) {
        const int64_t tiles = gemm_most_tiles(a, D == kWgrad, kBM);
        if (tiles * a.split > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
        return launch_gemm_as<2 * D + 1>(gemm_split_kernel<D, Few>, kSplitSmemMax, (unsigned)(tiles * a.split), kSplitThreads,
                              (unsigned)a.split, stream, maps, a, few);
    }
    const int64_t tiles = gemm_most_tiles(a, D == kWgrad, 2 * kBM), pairs = sm_count() / 2;
    return launch_gemm_as<2 * D>(gemm_kernel<D, Wide>, D == kWgrad ? kWgradSmemMax : kGemmSmemMax, 2u * (unsigned)(tiles < pairs ? tiles : pairs),
                          128 + 32 * Wide::kWarps, 2, stream,
                          maps, a, wide);
}

}  // namespace ep
