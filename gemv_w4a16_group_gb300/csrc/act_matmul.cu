// Products of quantized activations by NVFP4 and MXFP4 weights on the block-scaled tensor pipe:
//
//   y[m, n] = (r[m] S) sum_b sx[m, b] sw[n, b] sum_{k in b} x[m, k] w[n, k]
//
// with E2M1 (or, for 8-bit activations, E4M3) elements and the blocks' scales multiplied by the
// tensor pipe itself (tcgen05.mma, block_scale): an MMA takes 128 rows of weights by up to 128
// rows of x and 64 values of k (32 with 8-bit x), the elements from shared memory, one scale per
// 16 or 32 of them and row from tensor memory, and adds in fp32.
#include "act.h"
#include "common.cuh"

namespace w4k {
namespace {

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
// `sf` is the first scale's byte in its 32-bit word.
template <int FORM>
__host__ __device__ constexpr uint32_t idesc_scaled(int m, int n, int sf) {
  // element types: kind::mxf4nvf4 E2M1 = 1; kind::mxf8f6f4 E4M3 = 0, E2M1 = 5 (a: weights)
  const uint32_t ta = FORM == kActMxfp8 ? 5u : 1u, tb = FORM == kActMxfp8 ? 0u : 1u;
  return (static_cast<uint32_t>(sf) << 4) | (ta << 7) | (tb << 10) |
         (static_cast<uint32_t>(n >> 3) << 17) | ((FORM == kActNvfp4 ? 0u : 1u) << 23) |
         (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}

template <int FORM>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FORM == kActNvfp4)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else if constexpr (FORM == kActMxfp4)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// A 512-byte scale tile (32 rows of 16 bytes) into 4 columns of all four lane quarters.
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Descriptor of a scale tile: no swizzle, 8-row atoms of 128 bytes.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  return d;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 peer_lds64(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
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
  static constexpr int kSteps = F::KS / F::KM;
  // bytes that a copy of weights counts: those of the 4-bit values, also where it widens them
  static constexpr uint32_t w_tx = FORM == kActMxfp8 ? 128 * 64 : 128 * 128;
  static constexpr uint32_t w_bytes = 128 * 128, x_bytes = NT * 128, s_bytes = kTiles * 512;
  static constexpr uint32_t stage_bytes = w_bytes + x_bytes + 2 * s_bytes;
  // two CTAs an SM
  static constexpr int kStages = (110 * 1024) / stage_bytes;
  static constexpr uint32_t x_off = kStages * w_bytes;
  static constexpr uint32_t sw_off = x_off + kStages * x_bytes;
  static constexpr uint32_t sx_off = sw_off + kStages * s_bytes;
  static constexpr uint32_t bar_off = sx_off + kStages * s_bytes;  // full, empty, done
  static constexpr uint32_t misc_off = bar_off + (2 * kStages + 1) * 8;
  static constexpr uint32_t total = misc_off + 16;
  static constexpr uint32_t alloc = total + 1024;
  // tensor memory: the accumulator, two sets of scale columns
  static constexpr uint32_t s_cols = 4 * kTiles;
  static constexpr uint32_t acc_cols = NT < 32 ? 32 : NT;
  static constexpr uint32_t need_cols = acc_cols + 4 * s_cols;
  static constexpr uint32_t tmem_cols = need_cols <= 64 ? 64 : need_cols <= 128 ? 128 : 256;
  static_assert(need_cols <= 256, "two CTAs share the tensor memory");
  static_assert(NT * 128 * 4 <= kStages * (w_bytes + x_bytes), "the partial tile reuses the ring");
  static_assert(alloc <= 113 * 1024, "two CTAs share the shared memory");
};
constexpr int kNarrowThreads = 192;  // four warps for the tile, one for copies, one for the MMAs

template <int FORM, int NT>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    act_narrow_kernel(const __grid_constant__ NarrowMaps maps, const ActMatmulArgs a, int splits) {
  using L = Narrow<FORM, NT>;
  using F = Form<FORM>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar_off);
  uint64_t* empty = full + S;
  uint64_t* done = empty + S;
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile uint32_t* abort_flag = holder + 1;
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
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();

  int issued = 0;  // stages whose copies this thread has issued
  if (warp == 4) {
    if (lane == 0) {
      const int tiles_all = (a.K + F::KT - 1) / F::KT;
      const uint8_t* sw = a.w_scales + static_cast<size_t>(n0 >> 7) * tiles_all * 512;
      const uint8_t* sx = a.x_scales + static_cast<size_t>(m0 >> 7) * tiles_all * 512;
      for (int i = 0; i < count; ++i) {
        const int s = i % S;
        if (i >= S && !mbar_wait_bounded(&empty[s], ((i / S) & 1u) ^ 1u, abort_flag, a.status,
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
    if (lane == 0) {
      for (int i = 0; i < count; ++i) {
        const int s = i % S;
        if (!mbar_wait_bounded(&full[s], (i / S) & 1u, abort_flag, a.status, a.wait_limit_ns)) break;
        tc_fence_after_sync();
        const int k0 = (first + i) * F::KS;
        const uint32_t cols = tmem + L::acc_cols + (i & 1) * 2 * L::s_cols;
        const uint32_t sw = smem_addr(smem + L::sw_off + s * L::s_bytes);
        const uint32_t sx = smem_addr(smem + L::sx_off + s * L::s_bytes);
#pragma unroll
        for (int t = 0; t < L::kTiles; ++t) {
          if (k0 + t * F::KT >= a.K) break;
          scales_to_tmem(cols + 4 * t, smem_desc_scales(sw + t * 512));
          scales_to_tmem(cols + L::s_cols + 4 * t, smem_desc_scales(sx + t * 512));
        }
        const uint32_t ws = smem_addr(smem + s * L::w_bytes);
        const uint32_t xs = smem_addr(smem + L::x_off + s * L::x_bytes);
        constexpr int per_tile = F::KT / F::KM;
#pragma unroll
        for (int j = 0; j < L::kSteps; ++j) {
          if (k0 + j * F::KM >= a.K) break;
          const int t = j / per_tile;
          const int sf = j % per_tile * (4 / per_tile);
          const uint32_t idesc = idesc_scaled<FORM>(128, NT, sf);
          mma_scaled<FORM>(tmem, smem_desc_kmajor_sw128(ws + j * 32),
                           smem_desc_kmajor_sw128(xs + j * 32), idesc, cols + 4 * t,
                           cols + L::s_cols + 4 * t, (i | j) != 0 ? 1u : 0u);
        }
        tc_commit(&empty[s]);
      }
      // whatever happened, every MMA issued here completes before the tile is read or freed
      tc_commit(done);
    }
  }
  __syncwarp();
  volatile uint32_t none = 0u;
  bool ok = mbar_wait_bounded(done, 0u, &none, a.status, a.wait_limit_ns);
  if (!ok || *abort_flag)  // a wait has run out: the copies in flight land before anything else
    for (int s = 0; s < S && s < issued; ++s) {
      const int last = issued - 1 - ((issued - 1 - s) % S);
      mbar_wait_bounded(&full[s], (last / S) & 1u, &none, a.status, a.wait_limit_ns);
    }
  __syncwarp();
  __syncthreads();
  ok = ok && *abort_flag == 0u;
  tc_fence_after_sync();

  const float wscale = FORM == kActNvfp4 ? __ldg(a.w_scale) : 1.f;
  const int rows = min(NT, a.M - m0);
  if (warp < 4) {
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float* parts = reinterpret_cast<float*>(smem);  // [NT][128]
    const int n = n0 + warp * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < NT && c < rows; c += 16) {
      uint32_t v[16];
      __syncwarp();
      tmem_ld_16cols(lane_base + c, v);
      tmem_ld_wait();
      if (splits > 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          parts[(c + j) * 128 + warp * 32 + lane] = count > 0 ? __uint_as_float(v[j]) : 0.f;
      } else if (ok && n < a.N) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < rows) {
            float f = __uint_as_float(v[j]);
            if constexpr (FORM == kActNvfp4) f *= __ldg(a.x_rows + m0 + c + j) * wscale;
            a.y[static_cast<size_t>(m0 + c + j) * a.N + n] =
                __bfloat16_as_ushort(__float2bfloat16_rn(f));
          }
      }
    }
  }
  if (splits > 1) {
    __syncwarp();
    cluster_sync_all();
    // pairs of columns; the cluster's CTAs take the pairs in turn
    const uint32_t base = smem_addr(smem);
    for (int p = part * kNarrowThreads + threadIdx.x; p < rows * 64;
         p += splits * kNarrowThreads) {
      const int j = p >> 6, c = (p & 63) * 2;
      float2 sum = make_float2(0.f, 0.f);
      for (int r = 0; r < splits; ++r) {
        const float2 v = peer_lds64(peer_addr(base + (j * 128 + c) * 4, r));
        sum.x += v.x;
        sum.y += v.y;
      }
      if constexpr (FORM == kActNvfp4) {
        const float f = __ldg(a.x_rows + m0 + j) * wscale;
        sum.x *= f;
        sum.y *= f;
      }
      uint16_t* out = a.y + static_cast<size_t>(m0 + j) * a.N + n0 + c;
      if (ok && n0 + c < a.N) out[0] = __bfloat16_as_ushort(__float2bfloat16_rn(sum.x));
      if (ok && n0 + c + 1 < a.N) out[1] = __bfloat16_as_ushort(__float2bfloat16_rn(sum.y));
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another reads its part
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::tmem_cols);
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
  int splits = 1;
  while (splits < 8 && tn * tm * (splits + 1) <= 2 * sms && stages >= 2 * (splits + 1)) ++splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tn), static_cast<unsigned>(tm),
                     static_cast<unsigned>(splits));
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = L::alloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(splits);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, a, splits);
}

template <int FORM>
cudaError_t launch_form(const ActMatmulArgs& a, cudaStream_t stream) {
  if (a.M <= 16) return launch_narrow<FORM, 16>(a, stream);
  if (a.M <= 32) return launch_narrow<FORM, 32>(a, stream);
  if (a.M <= 64) return launch_narrow<FORM, 64>(a, stream);
  return launch_narrow<FORM, 128>(a, stream);
}

}  // namespace

cudaError_t launch_act_matmul(const ActMatmulArgs& a, int format, cudaStream_t stream) {
  if (format == kActNvfp4) return launch_form<kActNvfp4>(a, stream);
  if (format == kActMxfp4) return launch_form<kActMxfp4>(a, stream);
  return launch_form<kActMxfp8>(a, stream);
}

}  // namespace w4k
