// Products of quantized activations by NVFP4 and MXFP4 weights on the block-scaled tensor pipe:
//
//   y[m, n] = (r[m] S) sum_b sx[m, b] sw[n, b] sum_{k in b} x[m, k] w[n, k]
//
// with E2M1 (or, for 8-bit activations, E4M3) elements and the blocks' scales multiplied by the
// tensor pipe itself (tcgen05.mma, block_scale): an MMA takes 128 rows of weights by up to 128
// rows of x (few rows), or 256 rows of x by 256 of weights (a pair of CTAs), and 64 values of k (32
// with 8-bit x), the elements from shared memory, one scale per 16 or 32 of them and row from tensor
// memory, and adds in fp32.
#include "act.h"
#include "common.cuh"

namespace w4k {
namespace {

// Launches are plain ones: a kernel begins when the one before it on its stream has ended. What a
// resident CTA waits for without a limit is its own cluster, which is placed as a whole, and its
// columns of tensor memory: two narrow CTAs' fit in an SM, a wide CTA has the SM's shared memory to
// itself.

// A stage is a 128-byte swizzle row of k per row: 256 E2M1 or 128 E4M3 values. TILES scale tiles
// (128 rows x 4 scales, 512 bytes) cover it; an MMA takes KM values, STEPS of them a stage.
template <int FORM>
struct Form;
template <>
struct Form<kActNvfp4> {
  static constexpr int KS = 256, KM = 64, KT = 64;  // KT: values of k a scale tile covers
};
template <>
struct Form<kActMxfp4> {
  static constexpr int KS = 256, KM = 64, KT = 128;
};
template <>
struct Form<kActMxfp8> {
  static constexpr int KS = 128, KM = 32, KT = 128;
};

// Instruction descriptor of the block-scaled kinds: fp32 accumulator, both operands K-major.
// (The first scale's byte in its 32-bit word goes into bits 4 and 29 on.) W_IS_A: the weights are
// the A operand.
template <int FORM, bool W_IS_A>
__host__ __device__ constexpr uint32_t idesc_scaled(int m, int n) {
  // element types: kind::mxf4nvf4 E2M1 = 1; kind::mxf8f6f4 E4M3 = 0, E2M1 = 5
  const uint32_t w = FORM == kActMxfp8 ? 5u : 1u, x = FORM == kActMxfp8 ? 0u : 1u;
  const uint32_t ta = W_IS_A ? w : x, tb = W_IS_A ? x : w;
  return (ta << 7) | (tb << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((FORM == kActNvfp4 ? 0u : 1u) << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Operands as the low words of shared-memory descriptors; the high words are the layout's.
// Neighbouring pieces differ by an addition to the low word, and the whole warp computes them, so
// that they stay in uniform registers: a product costs its issuing warp a few instructions.
constexpr uint32_t kDescSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);  // see smem_desc_kmajor_sw128
// A scale tile: no swizzle, 8-row atoms of 128 bytes.
constexpr uint32_t kDescScales = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_low(const void* smem) {
  return (smem_addr(smem) & 0x3FFFFu) >> 4;
}

#define W4K_MMA_SCALED(GROUP, KIND)                                                              \
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\t"              \
               "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"                              \
               "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a, b, %3, [%4], [%5], "    \
               "p;\n\t}" ::"r"(d),                                                               \
               "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescSw128)  \
               : "memory")

// D (+)= A B with the scales at sfa and sfb; GROUP: the CTAs of a pair that hold the operands.
template <int FORM, int GROUP>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FORM == kActNvfp4) {
    if constexpr (GROUP == 1) W4K_MMA_SCALED("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else W4K_MMA_SCALED("2", "mxf4nvf4.block_scale.scale_vec::4X");
  } else if constexpr (FORM == kActMxfp4) {
    if constexpr (GROUP == 1) W4K_MMA_SCALED("1", "mxf4nvf4.block_scale.scale_vec::2X");
    else W4K_MMA_SCALED("2", "mxf4nvf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (GROUP == 1) W4K_MMA_SCALED("1", "mxf8f6f4.block_scale.scale_vec::1X");
    else W4K_MMA_SCALED("2", "mxf8f6f4.block_scale.scale_vec::1X");
  }
}
#undef W4K_MMA_SCALED

// A 512-byte scale tile (32 rows of 16 bytes) into 4 columns of all four lane quarters; a pair's
// CTAs each from their own shared memory into their own tensor memory.
template <int GROUP>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t desc) {
  if constexpr (GROUP == 1)
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(desc), "n"(kDescScales)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(desc), "n"(kDescScales)
        : "memory");
}

// mbar_wait_bounded for stages that change hands every few hundred nanoseconds: without a hint to
// suspend, and with the clock, whose reading takes longer than most waits, first read after some
// tries.
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t parity,
                                           volatile uint32_t* abort_flag, uint32_t* status,
                                           uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 31u) != 0) continue;
    if (*abort_flag) return false;
    const uint64_t t = global_timer_ns();
    if (t0 == 0) {
      t0 = t;
    } else if (t - t0 > limit_ns) {
      *abort_flag = 1u;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// How long a CTA that has given up a wait stays for its products and copies that are under way
// (microseconds in truth), whatever the limit of the waits themselves is.
constexpr uint64_t kSettleNs = 1000ull * 1000ull * 1000ull;

// One stage's scales and products: `a` and `b` the operands' tiles, sa and sb their scale tiles
// (low words of descriptors), BLOCKS_B row blocks of b's scales; columns of the scales in tensor
// memory at ca and cb. (Tiles begin at a block of 128 rows: scales that begin at an odd column
// fault.) WHOLE: all of the stage's k lies in the row; else `left` values of it.
template <int FORM, int GROUP, int BLOCKS_B, bool WHOLE>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t a, uint32_t b, uint32_t sa,
                                            uint32_t sb, uint32_t ca, uint32_t cb, uint32_t idesc,
                                            bool first, int left) {
  using F = Form<FORM>;
  constexpr int kTiles = F::KS / F::KT, kSteps = F::KS / F::KM, per_tile = F::KT / F::KM;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    if (!WHOLE && t * F::KT >= left) break;
    scales_to_tmem<GROUP>(ca + 4 * t, sa + t * 32);
#pragma unroll
    for (int blk = 0; blk < BLOCKS_B; ++blk)
      scales_to_tmem<GROUP>(cb + 4 * (t * BLOCKS_B + blk), sb + (blk * kTiles + t) * 32);
  }
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    if (!WHOLE && j * F::KM >= left) break;
    const int t = j / per_tile;
    const uint32_t sf = j % per_tile * (4 / per_tile);  // first scale's byte of the step
    mma_scaled<FORM, GROUP>(d, a + 2 * j, b + 2 * j, idesc | (sf << 4) | (sf << 29), ca + 4 * t,
                            cb + 4 * t * BLOCKS_B, !first || j != 0 ? 1u : 0u);
  }
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t peer_lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrives on the barrier at this address of CTA `rank` of the cluster.
__device__ __forceinline__ void peer_arrive(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                   peer_addr(smem_addr(bar), rank))
               : "memory");
}
// Tile load into this CTA's shared memory that completes on a barrier of either CTA of the pair
// (its shared::cluster address). x (innermost) must be a multiple of 16 bytes.
__device__ __forceinline__ void pair_load_2d(void* smem_dst, const CUtensorMap* map,
                                             uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(void* smem_dst, const CUtensorMap* map,
                                             uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Arrives (once) on `bar` of the pair's two CTAs (a bit each in `mask`, by rank in the cluster)
// when every MMA issued before has completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* smem_src, int x,
                                             int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::
                   "l"(reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(smem_src)), "r"(x), "r"(y)
               : "memory");
}

// What a row's sums are multiplied by, one factor after the other: r S and 1, or r and S where r S
// is at or past the ends of fp32's range (rows of 2^-60 by weights of 2^-60, say), though the sum times
// both need not be. Sums are 0 or 2^-20 to 2^46, act_quantize's r is 2^-92 to 2^117: sum r is then in
// range, or the result is not.
struct RowFactors {
  float f, g;
  __device__ __forceinline__ float of(float v) const { return v * f * g; }
};
__device__ __forceinline__ RowFactors row_factors(float r, float S) {
  const float f = r * S;
  return (f >= 0x1p-100f && f < 0x1p120f) || S == 0.f ? RowFactors{f, 1.f} : RowFactors{r, S};
}

// bf16(v f) to four columns of y, `left` of them inside it.
__device__ __forceinline__ void store_four(uint16_t* out, int left, int N, float4 v,
                                           RowFactors f) {
  if (left <= 0) return;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(f.of(v.x), f.of(v.y));
  const __nv_bfloat162 hi = __floats2bfloat162_rn(f.of(v.z), f.of(v.w));
  const uint2 w = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                             *reinterpret_cast<const uint32_t*>(&hi));
  if (N % 4 == 0) {
    *reinterpret_cast<uint2*>(out) = w;
  } else {
    out[0] = static_cast<uint16_t>(w.x);
    if (left > 1) out[1] = static_cast<uint16_t>(w.x >> 16);
    if (left > 2) out[2] = static_cast<uint16_t>(w.y);
    if (left > 3) out[3] = static_cast<uint16_t>(w.y >> 16);
  }
}

struct NarrowMaps {
  CUtensorMap w, x;
};

// Few rows of x: D is y's transpose. The MMA's A operand is 128 rows of weights (D's lanes are
// columns n of y), B is NT rows of x; a cluster of S CTAs shares a tile, each with its part of k,
// and adds the parts up through distributed shared memory in the CTAs' order.
template <int FORM, int NT>
struct Narrow {
  using F = Form<FORM>;
  static constexpr int kTiles = F::KS / F::KT;
  // bytes that a copy of weights counts: those of the 4-bit values, also where it widens them
  static constexpr uint32_t w_tx = FORM == kActMxfp8 ? 128 * 64 : 128 * 128;
  static constexpr uint32_t w_bytes = 128 * 128, x_bytes = NT * 128, s_bytes = kTiles * 512;
  static constexpr uint32_t stage_bytes = w_bytes + x_bytes + 2 * s_bytes;
  // Parts of a shared tile: up to 32 rows a CTA sends its sums to the CTA that adds them up, into
  // a place of their own, once its MMAs are done; more rows would cost stages, and are read from
  // where the sender's stages were.
  static constexpr bool kSend = NT <= 32;
  static constexpr uint32_t part_bytes = kSend ? NT * 128 * 4 : 0;
  // two CTAs an SM
  static constexpr int kStages = (112 * 1024 - part_bytes) / stage_bytes;
  static constexpr uint32_t x_off = kStages * w_bytes;
  static constexpr uint32_t sw_off = x_off + kStages * x_bytes;
  static constexpr uint32_t sx_off = sw_off + kStages * s_bytes;
  static constexpr uint32_t part_off = sx_off + kStages * s_bytes;
  static constexpr uint32_t bar_off = part_off + part_bytes;  // full, empty, done
  static constexpr uint32_t misc_off = bar_off + (2 * kStages + 1) * 8;
  static constexpr uint32_t whole_off = misc_off + 8;  // a word of each CTA of the cluster
  static constexpr uint32_t alloc = whole_off + 8 * 4;
  // tensor memory: the accumulator, two sets of scale columns
  static constexpr uint32_t s_cols = 4 * kTiles;
  static constexpr uint32_t acc_cols = NT < 32 ? 32 : NT;
  static constexpr uint32_t need_cols = acc_cols + 4 * s_cols;
  static constexpr uint32_t tmem_cols = need_cols <= 64 ? 64 : need_cols <= 128 ? 128 : 256;
  static_assert(need_cols <= 256, "two CTAs share the tensor memory");
  static_assert(kSend || NT * 128 * 4 <= kStages * (w_bytes + x_bytes), "parts reuse the ring");
  static_assert(alloc <= 113 * 1024, "two CTAs share the shared memory");
};
constexpr int kThreads = 192;  // four warps for the tile, one for copies, one for the MMAs

template <int FORM, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    act_narrow_kernel(const __grid_constant__ NarrowMaps maps, const ActMatmulArgs a, int splits) {
  using L = Narrow<FORM, NT>;
  using F = Form<FORM>;
  constexpr int S = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_addr(smem) & 1023u) != 0) {  // the same in every CTA
    if (threadIdx.x == 0) atomicOr(a.status, kStatusLayout);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar_off);
  uint64_t* empty = full + S;
  uint64_t* done = empty + S;
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile uint32_t* abort_flag = holder + 1;
  uint32_t* whole = reinterpret_cast<uint32_t*>(smem + L::whole_off);  // whether its sums are
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * 128, m0 = blockIdx.y * NT;
  const int part = blockIdx.z;  // this CTA's rank in its cluster

  const int stages_all = (a.K + F::KS - 1) / F::KS;
  const int per = (stages_all + splits - 1) / splits;
  const int first = part * per, count = max(0, min(stages_all, first + per) - first);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x);
  }
  if (warp == 5) {
    tmem_alloc(holder, L::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *holder;
  __syncwarp();
  // (waited for before anything is sent: every CTA of the cluster has begun)
  if (splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int rows = min(NT, a.M - m0);
  // a CTA of a cluster adds up 2^shift columns of the tile
  const int shift = 8 - __ffs(splits);
  const float wscale = FORM == kActNvfp4 ? __ldg(a.w_scale) : 1.f;
  // the row's scale of the first sums that this thread rounds
  const int j0 = static_cast<int>(threadIdx.x) >> (shift - 1);
  const float f0 = FORM == kActNvfp4 && j0 < rows ? __ldg(a.x_rows + m0 + j0) : 1.f;

  int issued = 0;  // stages whose copies this thread has issued
  if (warp == 4) {
    if (lane == 0) {
      const int tiles_all = (a.K + F::KT - 1) / F::KT;
      const uint8_t* sw = a.w_scales + static_cast<size_t>(n0 >> 7) * tiles_all * 512;
      const uint8_t* sx = a.x_scales + static_cast<size_t>(m0 >> 7) * tiles_all * 512;
      for (int i = 0; i < count; ++i) {
        const int s = i % S;
        if (i >= S && !stage_wait(&empty[s], ((i / S) & 1u) ^ 1u, abort_flag, a.status,
                                  a.wait_limit_ns))
          break;
        const int t0 = (first + i) * L::kTiles;
        const uint32_t sb = static_cast<uint32_t>(min(L::kTiles, tiles_all - t0)) * 512u;
        mbar_arrive_expect_tx(&full[s], L::w_tx + L::x_bytes + 2 * sb);
        // x coordinates: bytes of E2M1 pairs, or values where the copy widens them to bytes
        tma_load_2d(smem + s * L::w_bytes, &maps.w, &full[s], (first + i) * 128, n0);
        tma_load_2d(smem + L::x_off + s * L::x_bytes, &maps.x, &full[s], (first + i) * 128, m0);
        bulk_load(smem + L::sw_off + s * L::s_bytes, sw + static_cast<size_t>(t0) * 512, sb,
                  &full[s]);
        bulk_load(smem + L::sx_off + s * L::s_bytes, sx + static_cast<size_t>(t0) * 512, sb,
                  &full[s]);
        ++issued;
      }
    }
  } else if (warp == 5) {
    // the whole warp walks the stages, one lane issues
    constexpr uint32_t idesc = idesc_scaled<FORM, true>(128, NT);
    const uint32_t w0 = desc_low(smem), x0 = desc_low(smem + L::x_off);
    const uint32_t sw0 = desc_low(smem + L::sw_off), sx0 = desc_low(smem + L::sx_off);
    for (int i = 0; i < count; ++i) {
      const int s = i % S;
      if (!__all_sync(0xffffffffu, stage_wait(&full[s], (i / S) & 1u, abort_flag, a.status,
                                              a.wait_limit_ns)))
        break;
      tc_fence_after_sync();
      const int left = a.K - (first + i) * F::KS;
      const uint32_t ca = tmem + L::acc_cols + (i & 1) * 2 * L::s_cols;
      const uint32_t aw = w0 + s * (L::w_bytes >> 4), ax = x0 + s * (L::x_bytes >> 4);
      const uint32_t as = sw0 + s * (L::s_bytes >> 4), bs = sx0 + s * (L::s_bytes >> 4);
      if (elect_one()) {
        if (left >= F::KS)
          issue_stage<FORM, 1, 1, true>(tmem, aw, ax, as, bs, ca, ca + L::s_cols, idesc, i == 0,
                                        left);
        else
          issue_stage<FORM, 1, 1, false>(tmem, aw, ax, as, bs, ca, ca + L::s_cols, idesc, i == 0,
                                         left);
        tc_commit(&empty[s]);
      }
      __syncwarp();
    }
    // whatever happened, every MMA issued here completes before the tile is read or freed
    if (elect_one()) tc_commit(done);
  }
  __syncwarp();
  bool ok = stage_wait(done, 0u, abort_flag, a.status, a.wait_limit_ns);
  if (!ok || *abort_flag) {
    // a wait has run out: products and copies that are under way end before anything else
    volatile uint32_t none = 0u;
    stage_wait(done, 0u, &none, a.status, kSettleNs);
    for (int s = 0; s < S && s < issued; ++s) {
      const int last = issued - 1 - ((issued - 1 - s) % S);
      stage_wait(&full[s], (last / S) & 1u, &none, a.status, kSettleNs);
    }
  }
  __syncwarp();
  ok = __syncthreads_and(ok && *abort_flag == 0u);
  tc_fence_after_sync();

  if (splits > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (static_cast<int>(threadIdx.x) < splits)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                       peer_addr(smem_addr(whole + part), threadIdx.x)),
                   "r"(ok ? 1u : 0u)
                   : "memory");
  }
  if (warp < 4) {
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float* parts = reinterpret_cast<float*>(smem);  // [NT][128]
    const int col = warp * 32 + lane, n = n0 + col;
    // the CTA that adds up this column's sums, and where it has this one's: [splits][NT][width]
    const uint32_t to = peer_addr(smem_addr(smem + L::part_off), col >> shift) +
                        4 * (((part * NT) << shift) + (col & ((1 << shift) - 1)));
#pragma unroll 1
    for (int c = 0; c < NT && c < rows; c += 16) {
      uint32_t v[16];
      __syncwarp();
      tmem_ld_16cols(lane_base + c, v);
      tmem_ld_wait();
      if (L::kSend && splits > 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < rows)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + ((c + j) << (shift + 2))),
                         "r"(count > 0 ? v[j] : 0u)
                         : "memory");
      } else if (splits > 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          parts[(c + j) * 128 + col] = count > 0 ? __uint_as_float(v[j]) : 0.f;
      } else if (ok && n < a.N) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < rows) {
            float f = __uint_as_float(v[j]);
            if constexpr (FORM == kActNvfp4)
              f = row_factors(__ldg(a.x_rows + m0 + c + j), wscale).of(f);
            a.y[static_cast<size_t>(m0 + c + j) * a.N + n] =
                __bfloat16_as_ushort(__float2bfloat16_rn(f));
          }
      }
    }
  }
  if (splits > 1) {
    __syncwarp();
    cluster_sync_all();
    // a tile is stored where the sums of all its parts are whole
    for (int r = 0; r < splits; ++r) ok = ok && whole[r] != 0u;
    if constexpr (L::kSend) {
      const float2* parts = reinterpret_cast<const float2*>(smem + L::part_off);
      const int half = shift - 1;  // pairs of columns
      float f = f0;
      for (int p = threadIdx.x; p < rows << half; p += kThreads) {
        const int j = p >> half, c = p & ((1 << half) - 1), n = n0 + (part << shift) + 2 * c;
        if (FORM == kActNvfp4 && p >= kThreads) f = __ldg(a.x_rows + m0 + j);
        float2 sum = make_float2(0.f, 0.f);
        for (int r = 0; r < splits; ++r) {
          const float2 v = parts[((r * NT + j) << half) + c];
          sum.x += v.x;
          sum.y += v.y;
        }
        if constexpr (FORM == kActNvfp4) {
          const RowFactors by = row_factors(f, wscale);
          sum = make_float2(by.of(sum.x), by.of(sum.y));
        }
        uint16_t* out = a.y + static_cast<size_t>(m0 + j) * a.N + n;
        if (!ok || n >= a.N) continue;
        if (a.N % 2 == 0) {
          const __nv_bfloat162 w = __floats2bfloat162_rn(sum.x, sum.y);
          *reinterpret_cast<__nv_bfloat162*>(out) = w;
        } else {
          out[0] = __bfloat16_as_ushort(__float2bfloat16_rn(sum.x));
          if (n + 1 < a.N) out[1] = __bfloat16_as_ushort(__float2bfloat16_rn(sum.y));
        }
      }
    } else {
      // four columns at a time; the cluster's CTAs take them in turn, with the loads of all parts
      // on their way together
      const uint32_t base = smem_addr(smem);
      for (int p = part * kThreads + threadIdx.x; p < rows * 32;
           p += splits * kThreads) {
        const int j = p >> 5, c = (p & 31) * 4, n = n0 + c;
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < splits) v[r] = peer_lds128(peer_addr(base + (j * 128 + c) * 4, r));
        float4 sum = v[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < splits) {
            sum.x += v[r].x;
            sum.y += v[r].y;
            sum.z += v[r].z;
            sum.w += v[r].w;
          }
        const RowFactors f = FORM == kActNvfp4 ? row_factors(__ldg(a.x_rows + m0 + j), wscale)
                                               : RowFactors{1.f, 1.f};
        if (ok) store_four(a.y + static_cast<size_t>(m0 + j) * a.N + n, a.N - n, a.N, sum, f);
      }
      __syncwarp();
      cluster_sync_all();  // no CTA leaves while another reads its part
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::tmem_cols);
  }
}

// Many rows of x: a pair of CTAs on one MMA of 256 rows of x (A, 128 a CTA, D's lanes) by 256
// columns (B, half of the weights' rows in either CTA's shared memory), so that an operand's
// byte feeds twice the products of one CTA's tile. Persistent pairs; the accumulator has two
// places, so that a tile's MMAs run while the last one's sums are scaled, rounded and stored.
// With fewer tiles than pairs, a cluster of SPLIT pairs shares a tile, each with its part of k, and
// adds the parts up through distributed shared memory in the pairs' order.
struct WideMaps {
  CUtensorMap w, x, sw, sx, y;
};

constexpr int kWideN = 256;  // columns of a tile

template <int FORM>
struct Wide {
  using F = Form<FORM>;
  static constexpr int kTiles = F::KS / F::KT;
  static constexpr int kBlocks = kWideN / 128;  // row blocks of the weights' scales
  static constexpr uint32_t x_bytes = 128 * 128, w_bytes = kWideN / 2 * 128;
  static constexpr uint32_t w_tx = FORM == kActMxfp8 ? w_bytes / 2 : w_bytes;
  static constexpr uint32_t s_bytes = kTiles * 512;
  static constexpr uint32_t stage_bytes = x_bytes + w_bytes + (1 + kBlocks) * s_bytes;
  static constexpr uint32_t tx_bytes = x_bytes + w_tx + (1 + kBlocks) * s_bytes;  // of a CTA
  // pieces of y on their way out, 32 rows by 64 columns: two a warp where that costs no stage
  static constexpr int kRoom = 227 * 1024 - 256;
  static constexpr int kStages = (kRoom - 4 * 4096) / static_cast<int>(stage_bytes);
  static constexpr int kOut =
      (kRoom - 2 * 4 * 4096) / static_cast<int>(stage_bytes) == kStages ? 2 : 1;
  static constexpr uint32_t out_bytes = 4 * kOut * 4096;
  static constexpr uint32_t w_off = kStages * x_bytes;
  static constexpr uint32_t out_off = w_off + kStages * w_bytes;
  static constexpr uint32_t sx_off = out_off + out_bytes;
  static constexpr uint32_t sw_off = sx_off + kStages * s_bytes;
  static constexpr uint32_t bar_off = sw_off + kStages * kBlocks * s_bytes;
  // full (both CTAs' copies, in the first), empty; the accumulators' full (2), empty (2); done
  static constexpr uint32_t misc_off = bar_off + (2 * kStages + 5) * 8;
  static constexpr uint32_t alloc = misc_off + 16;
  static_assert(alloc <= 227 * 1024, "shared memory");
  // Tensor memory: the scales, and two accumulators, which overlap, since 512 columns do not hold
  // them apart; a tile's epilogue empties the columns that they share first.
  static constexpr uint32_t s_cols = 4 * kTiles * (1 + kBlocks);
  static constexpr uint32_t acc_step = (512 - kWideN - s_cols) / 64 * 64;
  static constexpr int kShared = (kWideN - static_cast<int>(acc_step)) / 64;  // 64-column pieces
  // a part of the sums between pairs: rows of floats, four apart in their banks
  static constexpr int kPartRow = kWideN + 4;
  static_assert(128 * kPartRow * 4 <= kStages * (x_bytes + w_bytes), "parts reuse the ring");
  static constexpr uint32_t sx_col = acc_step + kWideN;
  static constexpr uint32_t sw_col = sx_col + 4 * kTiles;
  static_assert(sx_col + s_cols <= 512, "tensor memory");
};

// Tiles in the order of their work: kGroup row tiles side by side, columns in turn, so that what
// the resident pairs read together stays in L2.
struct WideOrder {
  int tm, tn;
  static constexpr int kGroup = 16;
  __device__ __forceinline__ void at(int i, int& m, int& n) const {
    const int per = kGroup * tn, g = i / per, r = i - g * per;
    const int rows = min(kGroup, tm - g * kGroup);
    n = r / rows;
    m = g * kGroup + r - n * rows;
  }
};

template <int FORM, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2 * SPLIT, 1, 1)
    act_wide_kernel(const __grid_constant__ WideMaps maps, const ActMatmulArgs a,
                    const WideOrder order, int use_store) {
  using L = Wide<FORM>;
  using F = Form<FORM>;
  constexpr int S = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];  // (no room to align it by hand)
  if ((smem_addr(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusLayout);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar_off);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile uint32_t* abort_flag = holder + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // rank in the pair; the pair's part of k, its first CTA and both as a mask
  const uint32_t rank = cluster_rank() & 1u, part = cluster_rank() >> 1, lead = 2 * part;
  const uint16_t both = static_cast<uint16_t>(3u << lead);
  const int first = blockIdx.x / (2 * SPLIT), step = gridDim.x / (2 * SPLIT);
  const int tiles = order.tm * order.tn;
  const int stages = (a.K + F::KS - 1) / F::KS;  // SPLIT at least: no part is empty
  const int begin = static_cast<int>(part) * stages / SPLIT;
  const int end = (static_cast<int>(part) + 1) * stages / SPLIT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);  // the epilogue's warps of both CTAs
    }
    mbar_init(done, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.sw);
    tma_prefetch_desc(&maps.sx);
    if (SPLIT == 1 && use_store) tma_prefetch_desc(&maps.y);
  }
  // Both CTAs have begun and their barriers stand. Tensor memory comes after that: the pair takes it
  // together, and a request that finds no peer yet is never answered (one CTA may begin later where
  // other kernels' CTAs leave the pair's SMs; chains on several streams stood still). Nor is it used
  // before both have it; the copies do not wait for that.
  __syncwarp();
  cluster_sync_all();
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(holder)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before_sync();
  cluster_arrive();
  uint32_t tmem = 0;
  if (warp != 4) {
    cluster_wait();
    tc_fence_after_sync();
    tmem = *holder;
  }

  if (warp == 4) {
    if (lane == 0) {
      const uint32_t full0 = peer_addr(smem_addr(full), lead);
      const int w_row = static_cast<int>(rank) * (kWideN / 2);
      int s = 0;
      uint32_t phase = 1;  // of the stage's last use
      bool go = true;
      for (int t = first; t < tiles && go; t += step) {
        int tm, tn;
        order.at(t, tm, tn);
        const int bm = tm * 2 + static_cast<int>(rank);
        for (int i = begin; i < end; ++i) {
          if (!stage_wait(&empty[s], phase, abort_flag, a.status, a.wait_limit_ns)) {
            go = false;
            break;
          }
          const uint32_t bar = full0 + s * 8;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::tx_bytes);
          // rows and scale tiles past the arrays come as zeros
          pair_load_2d(smem + s * L::x_bytes, &maps.x, bar, i * 128, bm * 128);
          pair_load_3d(smem + L::sx_off + s * L::s_bytes, &maps.sx, bar, 0, i * L::kTiles, bm);
          pair_load_2d(smem + L::w_off + s * L::w_bytes, &maps.w, bar, i * 128, tn * kWideN + w_row);
          pair_load_3d(smem + L::sw_off + s * L::kBlocks * L::s_bytes, &maps.sw, bar, 0,
                       i * L::kTiles, tn * L::kBlocks);
          if (++s == S) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
    cluster_wait();  // (of the arrival above)
  } else if (warp == 5 && rank == 0) {
    // the whole warp walks the stages, one lane issues the pair's MMAs
    constexpr uint32_t idesc = idesc_scaled<FORM, false>(256, kWideN);
    const uint32_t x0 = desc_low(smem), w0 = desc_low(smem + L::w_off);
    const uint32_t sx0 = desc_low(smem + L::sx_off), sw0 = desc_low(smem + L::sw_off);
    const uint32_t ca = tmem + L::sx_col, cb = tmem + L::sw_col;
    int s = 0, n_tile = 0;
    uint32_t phase = 0;
    bool go = true;
    for (int t = first; t < tiles && go; t += step, ++n_tile) {
      const int b = n_tile & 1;
      const uint32_t acc = tmem + b * L::acc_step;
      if (n_tile > 0) {
        const int q = n_tile - 1;  // the tile whose shared columns must be empty
        go = __all_sync(0xffffffffu, stage_wait(&acc_empty[q & 1], (q >> 1) & 1u, abort_flag,
                                                a.status, a.wait_limit_ns));
        if (!go) break;
        tc_fence_after_sync();
      }
      for (int i = begin; i < end; ++i) {
        go = __all_sync(0xffffffffu,
                        stage_wait(&full[s], phase, abort_flag, a.status, a.wait_limit_ns));
        if (!go) break;
        tc_fence_after_sync();
        const int left = a.K - i * F::KS;
        const uint32_t ax = x0 + s * (L::x_bytes >> 4), bw = w0 + s * (L::w_bytes >> 4);
        const uint32_t as = sx0 + s * (L::s_bytes >> 4);
        const uint32_t bs = sw0 + s * (L::kBlocks * L::s_bytes >> 4);
        if (elect_one()) {
          if (left >= F::KS)
            issue_stage<FORM, 2, L::kBlocks, true>(acc, ax, bw, as, bs, ca, cb, idesc, i == begin,
                                                   left);
          else
            issue_stage<FORM, 2, L::kBlocks, false>(acc, ax, bw, as, bs, ca, cb, idesc, i == begin,
                                                    left);
          pair_commit(&empty[s], both);
          if (i == end - 1) pair_commit(&acc_full[b], both);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    if (elect_one()) pair_commit(done, both);
  } else if (warp < 4) {
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float wscale = FORM == kActNvfp4 ? __ldg(a.w_scale) : 1.f;
    uint8_t* out = smem + L::out_off + warp * (L::kOut * 4096);
    int n_tile = 0, piece = 0;
    for (int t = first; t < tiles; t += step, ++n_tile) {
      const int b = n_tile & 1;
      int tm, tn;
      order.at(t, tm, tn);
      const int row0 = tm * 256 + static_cast<int>(rank) * 128 + warp * 32;
      const int row = row0 + lane;
      RowFactors f = {1.f, 1.f};
      if constexpr (FORM == kActNvfp4)
        f = row_factors(row < a.M ? __ldg(a.x_rows + row) : 0.f, wscale);
      bool ok = stage_wait(&acc_full[b], (n_tile >> 1) & 1u, abort_flag, a.status,
                           a.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
#pragma unroll 1
      for (int cc = 0; cc < kWideN / 64; ++cc) {
        // the columns that the other accumulator shares come first
        const int c = b == 0 ? kWideN / 64 - 1 - cc : cc;
        uint32_t v[64];
        tmem_ld_32cols(lane_base + b * L::acc_step + c * 64, v);
        tmem_ld_32cols(lane_base + b * L::acc_step + c * 64 + 32, v + 32);
        tmem_ld_wait();
        if (cc == L::kShared - 1) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) peer_arrive(&acc_empty[b], lead);
        }
        if constexpr (SPLIT > 1) {
          // the pair's part of the sums, where its stages were
          float4* to =
              reinterpret_cast<float4*>(smem) + (warp * 32 + lane) * (L::kPartRow / 4) + c * 16;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            to[j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          continue;
        }
        const int n0 = tn * kWideN + c * 64;
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float lo = __uint_as_float(v[2 * j]), hi = __uint_as_float(v[2 * j + 1]);
          if constexpr (FORM == kActNvfp4) {
            lo = f.of(lo);
            hi = f.of(hi);
          }
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[j]) : "f"(hi), "f"(lo));
        }
        if (use_store) {
          // a piece of 32 rows by 64 columns through shared memory (128-byte swizzle)
          if (row0 < a.M && n0 < a.N) {  // warp-uniform
            uint8_t* dst = out + piece * 4096;
            if constexpr (L::kOut == 2) piece ^= 1;
            if (lane == 0)
              asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(L::kOut - 1) : "memory");
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(dst + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                  make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.y, dst, n0, row0);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        } else if (row < a.M) {  // rows of y that are not 16-byte aligned
          uint16_t* dst = a.y + static_cast<size_t>(row) * a.N;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (n0 + 2 * j < a.N) dst[n0 + 2 * j] = static_cast<uint16_t>(p[j]);
            if (n0 + 2 * j + 1 < a.N) dst[n0 + 2 * j + 1] = static_cast<uint16_t>(p[j] >> 16);
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  volatile uint32_t none = 0u;
  // (a warp without a part in the work does not wait for all of it, which may pass the limit)
  const bool idle = warp == 5 && rank != 0;
  if (!idle && (!stage_wait(done, 0u, &none, a.status, a.wait_limit_ns) || *abort_flag)) {
    // a wait has run out: products and copies under way (microseconds) end before anything else; a
    // fixed time, since the first CTA's barriers, on which copies end, count both CTAs' whole stages
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000u) {
    }
  }
  tc_fence_before_sync();
  __syncwarp();
  if constexpr (SPLIT > 1) {
    cluster_sync_all();  // the parts stand
    int tm, tn;
    order.at(first, tm, tn);
    // stored where the sums of all pairs are whole
    bool ok = true;
#pragma unroll
    for (int p = 0; p < SPLIT; ++p)
      ok = ok && peer_lds32(peer_addr(smem_addr(holder + 1), 2 * p + rank)) == 0u;
    const float wscale = FORM == kActNvfp4 ? __ldg(a.w_scale) : 1.f;
    const uint32_t base = smem_addr(smem);
    // this pair's share of the columns, four at a time; neighbouring threads take neighbours, and
    // the loads of kBatch turns are on their way together
    constexpr int kQuads = kWideN / SPLIT / 4, kBatch = 4;
    for (int q0 = threadIdx.x; q0 < 128 * kQuads; q0 += kBatch * kThreads) {
      float4 v[kBatch][SPLIT];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int q = min(q0 + u * kThreads, 128 * kQuads - 1), r = q / kQuads;
        const int c = (static_cast<int>(part) * kQuads + q % kQuads) * 4;
#pragma unroll
        for (int p = 0; p < SPLIT; ++p)
          v[u][p] = peer_lds128(peer_addr(base + (r * L::kPartRow + c) * 4, 2 * p + rank));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int q = q0 + u * kThreads, r = q / kQuads;
        const int c = (static_cast<int>(part) * kQuads + q % kQuads) * 4;
        const int row = tm * 256 + static_cast<int>(rank) * 128 + r, n = tn * kWideN + c;
        if (!ok || q >= 128 * kQuads || row >= a.M || n >= a.N) continue;
        float4 sum = v[u][0];
#pragma unroll
        for (int p = 1; p < SPLIT; ++p) {
          sum.x += v[u][p].x;
          sum.y += v[u][p].y;
          sum.z += v[u][p].z;
          sum.w += v[u][p].w;
        }
        RowFactors f = {1.f, 1.f};
        if constexpr (FORM == kActNvfp4) f = row_factors(__ldg(a.x_rows + row), wscale);
        store_four(a.y + static_cast<size_t>(row) * a.N + n, a.N - n, a.N, sum, f);
      }
    }
    __syncwarp();
  }
  cluster_sync_all();  // neither CTA leaves while the other's MMAs or arrivals reach it
  if (warp == 5) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

// Rows of `K` values as the copies see them: bytes (E2M1 pairs, E4M3), or 4-bit values that the
// copy widens to a byte each (16 values in the first 8 of 16 bytes, the form kind::mxf8f6f4 reads).
cudaError_t make_map(CUtensorMap* map, const uint8_t* codes, int rows, int K, int box_rows,
                     bool bytes, bool widen) {
  if (widen)
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, codes,
                             static_cast<uint64_t>(K), static_cast<uint64_t>(rows),
                             static_cast<uint64_t>(K) / 2, 128, static_cast<uint32_t>(box_rows),
                             CU_TENSOR_MAP_SWIZZLE_128B);
  const uint64_t row = bytes ? static_cast<uint64_t>(K) : static_cast<uint64_t>(K) / 2;
  return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, row,
                           static_cast<uint64_t>(rows), row, 128, static_cast<uint32_t>(box_rows),
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int FORM, int NT>
cudaError_t launch_narrow(const ActMatmulArgs& a, cudaStream_t stream) {
  using L = Narrow<FORM, NT>;
  using F = Form<FORM>;
  NarrowMaps maps;
  constexpr bool x8 = FORM == kActMxfp8;
  cudaError_t e = make_map(&maps.w, a.w_codes, a.N, a.K, 128, false, x8);
  if (e != cudaSuccess) return e;
  e = make_map(&maps.x, a.x_codes, a.M, a.K, NT, x8, false);
  if (e != cudaSuccess) return e;
  auto kern = act_narrow_kernel<FORM, NT>;
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(L::alloc));
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long tn = (a.N + 127) / 128, tm = (a.M + NT - 1) / NT;
  if (tm > 65535) return cudaErrorInvalidConfiguration;
  const int stages = (a.K + F::KS - 1) / F::KS;
  // As many CTAs a tile as the SMs hold at once, two each (clusters of 4 and 8 leave some SMs of a
  // GPC without: 74 and 36 fit on 152 SMs), with two stages each at least. Powers of two: 48
  // tiles took 22 us with clusters of 6, two waves of them, and 18 with 4.
  int splits = 8;
  while (splits > 1 &&
         (stages < 2 * splits || tn * tm > 2 * sms / splits - (splits > 2 ? 2 : 0)))
    splits /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tn), static_cast<unsigned>(tm),
                     static_cast<unsigned>(splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::alloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(splits);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, a, splits);
}

// Scale tiles: 512 bytes (128 words), tiles along k, row blocks.
cudaError_t make_scale_map(CUtensorMap* map, const uint8_t* scales, int rows, int tiles_k,
                           int box_tiles, int box_blocks) {
  const uint64_t dims[3] = {128, static_cast<uint64_t>(tiles_k),
                            (static_cast<uint64_t>(rows) + 127) / 128};
  const uint64_t strides[2] = {512, static_cast<uint64_t>(tiles_k) * 512};
  const uint32_t box[3] = {128, static_cast<uint32_t>(box_tiles),
                           static_cast<uint32_t>(box_blocks)};
  return encode_tensor_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_INT32, scales, dims, strides, box,
                              CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int FORM, int SPLIT>
cudaError_t launch_wide(const ActMatmulArgs& a, cudaStream_t stream) {
  using L = Wide<FORM>;
  WideMaps maps = {};
  constexpr bool x8 = FORM == kActMxfp8;
  cudaError_t e = make_map(&maps.w, a.w_codes, a.N, a.K, kWideN / 2, false, x8);
  if (e != cudaSuccess) return e;
  e = make_map(&maps.x, a.x_codes, a.M, a.K, 128, x8, false);
  if (e != cudaSuccess) return e;
  const int tiles_k = (a.K + Form<FORM>::KT - 1) / Form<FORM>::KT;
  e = make_scale_map(&maps.sx, a.x_scales, a.M, tiles_k, L::kTiles, 1);
  if (e != cudaSuccess) return e;
  e = make_scale_map(&maps.sw, a.w_scales, a.N, tiles_k, L::kTiles, L::kBlocks);
  if (e != cudaSuccess) return e;
  // (sums of several parts are stored from registers)
  const int use_store = SPLIT == 1 && a.N % 8 == 0;
  if (use_store) {
    e = encode_tensor_map(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.y, static_cast<uint64_t>(a.N),
                          static_cast<uint64_t>(a.M), static_cast<uint64_t>(a.N) * 2, 64, 32,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  auto kern = act_wide_kernel<FORM, SPLIT>;
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(L::alloc));
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const WideOrder order = {(a.M + 255) / 256, (a.N + kWideN - 1) / kWideN};
  const long long tiles = static_cast<long long>(order.tm) * order.tn;
  if (tiles > 0x7fffffffLL - 2 * sms) return cudaErrorInvalidConfiguration;
  const int clusters = static_cast<int>(SPLIT > 1 || tiles < sms / 2 ? tiles : sms / 2);
  kern<<<static_cast<unsigned>(2 * SPLIT * clusters), kThreads, L::alloc, stream>>>(maps, a, order,
                                                                                    use_store);
  return cudaGetLastError();
}

template <int FORM>
cudaError_t launch_form(const ActMatmulArgs& a, int kernel, cudaStream_t stream) {
  const int stages = (a.K + Form<FORM>::KS - 1) / Form<FORM>::KS;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long tiles =
      ((static_cast<long long>(a.M) + 255) / 256) * ((static_cast<long long>(a.N) + 255) / 256);
  if (kernel == 0) {
    // The pairs' tiles of 256 x 256 want 256 rows of x or enough columns: 14336 x 4096 NVFP4 at 64
    // rows 12.1 us (narrow 12.7), at 56 12.4 either way, at 48 12.7 (11.9), MXFP8 at 96 15.6 (15.8), at
    // 80 15.5 (15.3), at 64 15.2 (13.1); 4096 x 14336 NVFP4 at 256 rows 19.5 (16.6), at 320 19.7
    // (21.4). (Of the narrow kernel's end at 256 rows: with few columns it would win a little longer,
    // 1536 x 8960 at 384 rows NVFP4 12.4 against 13.7 of four pairs a tile, MXFP8 13.8 against 15.3.)
    const int few = FORM == kActMxfp8 ? 80 : 48;
    kernel = a.M <= few || (a.M <= 256 && tiles * 5 < sms) ? 1 : 2;
    // With few tiles pairs share them, where each part of k outweighs adding the parts up (4096 x
    // 14336 MXFP4 at 512 rows 21.8 -> 17.2 us with two a tile, 1536 x 8960 MXFP8 at 384 25.1 -> 17.3 with
    // two, 15.3 with four; 16 stages are even). 36 clusters of two pairs and 15 of four fit on 152 SMs.
    if (kernel == 2 && stages >= 24)
      kernel = tiles * 10 <= sms ? 4 : tiles * 4 <= sms - 8 ? 3 : 2;
  }
  if (kernel == 4 && stages >= 4) return launch_wide<FORM, 4>(a, stream);
  if (kernel >= 3 && stages >= 2) return launch_wide<FORM, 2>(a, stream);
  if (kernel >= 2) return launch_wide<FORM, 1>(a, stream);
  if (a.M <= 16) return launch_narrow<FORM, 16>(a, stream);
  if (a.M <= 32) return launch_narrow<FORM, 32>(a, stream);
  if (a.M <= 64) return launch_narrow<FORM, 64>(a, stream);
  return launch_narrow<FORM, 128>(a, stream);
}

}  // namespace

cudaError_t launch_act_matmul(const ActMatmulArgs& a, int format, int kernel, cudaStream_t stream) {
  if (format == kActNvfp4) return launch_form<kActNvfp4>(a, kernel, stream);
  if (format == kActMxfp4) return launch_form<kActMxfp4>(a, kernel, stream);
  return launch_form<kActMxfp8>(a, kernel, stream);
}

}  // namespace w4k
