// Attention of a few new tokens over the 4-bit key/value cache.
//
//   s_ij = scale q_i . k_hat_j (j <= n - m + i),  p = softmax_j(s),  out_i = sum_j p_ij v_hat_j
//
// Rows are the (new token, query head) pairs that share a key/value head, 8 NT of them a tile.
// With c the code, s the scale and m the minimum of a dim's group g,
//   q . k_hat_j = sum_g s_jg (sum_{d in g} q_d c_jd) + m_jg (sum_{d in g} q_d)
//   sum_j p_j v_hat_jd = sum_j (p_j s_jg) c_jd + sum_j p_j m_jg
// so the codes go to the tensor pipe as they are, and the scales touch one number a token and
// group. A code masked out of its word is an FP16 subnormal, a power of two times the code, which
// the MMA multiplies exactly: five or six operations for eight codes. (128 + c or 1024 + c needs
// the offset's sum taken out again; the MMA truncates its sums, and over 131072 tokens the offset,
// hundreds of times the result, cost 1.2 % of it. Centring the pairs cures that for four more
// operations.) q is FP16 under a power of two a row, exact down to 2^-27 of the row's largest; p s
// is rounded to FP16 under a power of two a row (2^-11 of itself or 2^-28 of the row's largest, see
// kLift; BF16's 2^-8 was twice the output's own rounding error). Sums, maxima and the softmax's
// statistics are fp32.
//
// What bounds it: the cache is read once (D + 8 D / group bytes a token and head), at 4 heads a
// key/value head about 8 operations a byte, so the aim is the memory's rate. 64 sequences of 8192
// tokens, 32 heads on 8 of 128: 604 MB of cache in 104.5 us, 5.8 TB/s (0.85 of a copy's rate), with
// weights 67 MB of logits more and read again, 130 us; one of 131072 tokens 32.0 us, 4.5 TB/s, of
// which some 7 us are the launch, the first copies and the join. Issue slots (48 % of cycles), ALU
// (48 %) and DRAM (60 %) are all half busy in 24 sequences of 8192: latency between the few warps
// that the accumulators leave room for.
//
// Work split. A unit is 32 tokens of one (sequence, head, row tile); the units of all sequences
// in order are cut into equal ranges, one a CTA, from the lengths on the device: ragged batches
// and one long sequence use the whole GPU alike, and a bound on the length costs nothing. Within
// a range the computing warps take units in turn, each from its own ring of bulk copies that
// one more warp keeps filled; there is no barrier but at a segment (the part of one sequence, head
// and tile in the range), whose rows one warp prepares and whose end joins the warps' (max, sum,
// accumulator) through shared memory. A segment that another CTA shares goes to the workspace in
// fp32, and the CTA that arrives last joins the parts in order. (Copies issued by the computing
// warps themselves, with a page looked up for each, cost them registers and a sixth of their
// instructions.)
#include <type_traits>

#include "kv4_common.cuh"
#include "kv4_prompt.h"

namespace w4k {
namespace {

// Computing warps of a CTA (with the copies' warp eight) and resident CTAs an SM, by what the
// accumulators of nt n8 tiles of rows leave of the registers: 128 a thread or all 255.
constexpr int kWarps = 7;
constexpr int ctas_per_sm(int d, int nt) { return d * nt <= 128 ? 2 : 1; }
// Copies a warp has on their way or at hand: what two CTAs' shared memory holds.
constexpr int ring_stages(int d, int ng) { return d == 128 && ng == 4 ? 2 : 3; }
constexpr int kUnit = 32;  // tokens
constexpr int kUnitRecords = kUnit / 16;
constexpr uint32_t kAllRecords = (1u << kUnitRecords) - 1u;
// Units that stand for what an item (sequence, head, row tile) costs beyond its own: loading its
// queries, joining the warps, writing its rows. They come before its units in the list. Without
// them the CTA that got the shortest sequences of a ragged batch (0, 1, 17 .. 4096 tokens, 32
// sequences of 8 heads) took 42 us, its neighbours 10. A unit is one of seven that run at once, so
// an item's 4 us are many. At 12 / 26 / 40, us: that batch 18.0 / 17.7 / 18.8, 16 sequences of 100
// to 16384 tokens 23.4 / 21.7 / 22.6, 8 of 300 to 8000 with 8 new tokens 37.8 / 34.6 / 32.5, 16 of
// 300 to 3001 with 5 (head size 64) 20.6 / 18.0 / 19.6, 64 of 8192 104.5 / 104.5 / 105.2.
constexpr int kItemCost = 26;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Probabilities times V scales, as the second product's FP16 operand. A row's products come under
// 2^-e, e the exponent of the largest one that it has met (at most 1 times a scale, while the
// running maximum is exact), and have these bits to spare above it: the running maximum lags by up
// to 2^kLag, a scale may be 2^kScaleLag times the largest product, and what is left lifts the
// products, so that they are rounded to 2^-11 of themselves or 2^-28 of the largest. (Under the
// largest scale that the row had met, attended or not, one token of values 2^20 times the others'
// took 20 bits of theirs.)
constexpr int kLag = 4, kScaleLag = 8, kLift = 15 - kLag - kScaleLag;
// The least e (exponent field): 2^kLag times 2^(127 + kLift - e) is still a number, and 0 times it
// 0 where a group's values are equal and their scale is 0.
constexpr int kLeastEv = 16;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// FP16 pairs of nibbles i and i + 4. The MMA lines its products up by their operands' exponent
// fields, so the zeros above a subnormal's bits are bits lost of the sum: the higher a code lies in
// the mantissa the better.
// Keys: q 2^-22 for even i, q 2^-18 for odd i (with q 2^-24 and q 2^-20, one shift less, the
// log-sums were off by 1e-6 of themselves, now by 1e-7).
__device__ __forceinline__ void key_pairs(uint32_t w, uint32_t (&p)[4]) {
  p[0] = (w << 2) & 0x003C003Cu;
  p[1] = (w << 2) & 0x03C003C0u;
  p[2] = (w >> 6) & 0x003C003Cu;
  p[3] = (w >> 6) & 0x03C003C0u;
}
// Values, where the output's rounding hides it: q 2^-24, 2^-20, 2^-22, 2^-18.
__device__ __forceinline__ void value_pairs(uint32_t w, uint32_t (&p)[4]) {
  p[0] = w & 0x000F000Fu;
  p[1] = w & 0x00F000F0u;
  p[2] = (w >> 6) & 0x003C003Cu;
  p[3] = (w >> 6) & 0x03C003C0u;
}

// D(16x8) = A(16x16) B(16x8), FP16 in, fp32 out.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <int NB>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t (&w)[NB]) {
  if constexpr (NB == 4) {
    const uint4 v = lds128(addr);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  }
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Barrier of the computing warps.
__device__ __forceinline__ void join_warps() {
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

// bulk_load of bytes that the call reads once and that leave L2 first: the logits stay (64
// sequences of 8192 with weights 135.8 -> 130.4 us, 16 of them 46 -> 41; without weights 106.8 ->
// 104.5; 4 of them, a cache that fits L2 and is read again at once, 15.5 either way).
__device__ __forceinline__ void bulk_load_once(void* smem_dst, const void* gsrc, uint32_t bytes,
                                               uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

struct Workspace {
  uint32_t* counters;  // [grid], of the item that a CTA's range begins and does not end
  float* lse2;         // [tokens, heads], base 2
  float* logits;       // [batch, kv_heads, max_new G, row_len], base 2 (weights only)
  float* parts;        // [2 grid] x (8 NT rows x D + 16 NT)
  int row_len;
};

// The units of sequence b: sequences without new tokens have none, an empty one has one a tile
// (its rows are still to be written).
struct Work {
  Kv4Seq s;
  int tiles, chunks;  // row tiles, units of each
};
template <int ROWS>
__device__ __forceinline__ Work work_of(const Kv4AttentionArgs& a, int group, int b) {
  Work w;
  w.s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
  w.tiles = (w.s.m * group + ROWS - 1) / ROWS;
  w.chunks = max(1, (w.s.n + kUnit - 1) / kUnit);
  return w;
}

// An item and its units in this CTA's range, a segment.
struct Cursor {
  int b, h, tile;
  Work w;
  int lo, hi;
  uint32_t base;  // the item's first place in the list
  uint32_t left;  // places of the range after this segment's
};

__device__ __forceinline__ void enter(Cursor& c, int first) {
  const int end =
      static_cast<int>(min(static_cast<uint32_t>(kItemCost + c.w.chunks), first + c.left));
  c.left -= end - first;
  c.lo = max(0, first - kItemCost);
  c.hi = max(0, end - kItemCost);
}

// Next segment of the range that has units (the range's end may hold only an item's cost); false
// at its end.
template <int ROWS>
__device__ __forceinline__ bool advance(Cursor& c, const Kv4AttentionArgs& a, int group) {
  do {
    if (c.left == 0) return false;
    c.base += kItemCost + c.w.chunks;
    if (++c.tile >= c.w.tiles) {
      c.tile = 0;
      if (++c.h >= a.c.kv_heads) {
        c.h = 0;
        do {
          if (++c.b >= a.c.batch) return false;
          c.w = work_of<ROWS>(a, group, c.b);
        } while (c.w.tiles == 0);
      }
    }
    enter(c, 0);
  } while (c.lo >= c.hi);
  return true;
}

// PACK: up to four rows stand in columns 0..3 for a unit's first record and again in 4..7 for its
// second, so that one accumulator holds the logits of both and every lane's share of the softmax
// is of use (otherwise half of the columns pad the tile).
template <int D, int NG, int NT, bool PACK>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStages = ring_stages(D, NG);
  static constexpr int kLower = (kWarps + 1) / 2;  // accumulators in shared memory at a time
  static_assert(!PACK || kWarps * 4 <= kLower * kRows, "packed: all warps' four rows");
  static constexpr uint32_t stage_bytes = kUnitRecords * Kv4Record<D, NG>::kBytes;
  // the queries, [nt][D / 32][lane] 16 bytes, until the warps join; then accumulators,
  // [kLower][row][D]
  static constexpr uint32_t q_off = kWarps * kStages * stage_bytes;
  static constexpr uint32_t o_off = q_off;
  static constexpr uint32_t ml_off = o_off + kLower * kRows * D * 4;  // [warp][row] (m, l)
  static constexpr uint32_t row_off = ml_off + kWarps * kRows * 8;   // [row] (sums of q, unscale)
  static constexpr uint32_t bar_off = row_off + kRows * (NG + 1) * 4;
  static constexpr uint32_t have_off = bar_off + 2 * kWarps * kStages * 8;  // [warp][stage]
  static constexpr uint32_t misc_off = have_off + kWarps * kStages * 4;
  static constexpr uint32_t total = misc_off + 16;
  static constexpr int part_floats = kRows * D + 2 * kRows;
  static_assert(total <= (ctas_per_sm(D, NT) == 2 ? 113u : 227u) * 1024u, "shared memory");
};

template <int D, int NG, int NT, bool PACK, bool LOGITS>
__global__ void __launch_bounds__((kWarps + 1) * 32, ctas_per_sm(D, NT))
    kv4_attention_kernel(const Kv4AttentionArgs a, const Workspace ws) {
  using R = Kv4Record<D, NG>;
  using S = Shape<D, NG, NT, PACK>;
  static_assert(!PACK || (NT == 1 && kUnitRecords == 2), "two records, eight columns");
  constexpr int NB = R::kBlocks, kRows = S::kRows, kLower = S::kLower, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::bar_off);  // [warp][stage]
  uint64_t* empty = full + kWarps * kStages;
  // bit j: a stage holds its unit's record j (not past the length, nor of a page out of range)
  volatile uint32_t* stage_has = reinterpret_cast<uint32_t*>(smem + S::have_off);
  volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + S::misc_off);
  volatile uint32_t* arrived = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.heads / a.c.kv_heads;

  if (threadIdx.x < 2 * kWarps * kStages) mbar_init(&full[threadIdx.x], 1);
  if (threadIdx.x == 0) *abort_flag = 0u;
  if (warp == 0) {
    __syncwarp();
    if (lane == 0) fence_barrier_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  // This CTA's range of units: lane by lane the sequences' units, and among them the range's
  // beginning.
  uint32_t total = 0;
  Work mine;
  auto units_of = [&](int b) {
    if (b >= a.c.batch) return 0u;
    mine = work_of<kRows>(a, G, b);
    return static_cast<uint32_t>(mine.tiles) * (kItemCost + mine.chunks) * a.c.kv_heads;
  };
  for (int base = 0; base < a.c.batch; base += 32)
    total += __reduce_add_sync(0xffffffffu, units_of(base + lane));
  const uint32_t ctas = min(gridDim.x, (total + kWarps - 1) / kWarps), me = blockIdx.x;
  if (me >= ctas) return;
  const Shares shares(total, ctas);
  const uint32_t u0 = shares.begin(me);

  Cursor cur;
  {
    uint32_t before = 0;
    for (int base = 0;; base += 32) {
      const uint32_t u = units_of(base + lane);
      uint32_t upto = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, u0 < before + upto);
      if (hit != 0) {
        const int at = __ffs(hit) - 1;
        before += __shfl_sync(0xffffffffu, upto - u, at);
        cur.b = base + at;
        cur.w.s.n = __shfl_sync(0xffffffffu, mine.s.n, at);
        cur.w.s.m = __shfl_sync(0xffffffffu, mine.s.m, at);
        cur.w.s.s0 = __shfl_sync(0xffffffffu, mine.s.s0, at);
        cur.w.tiles = __shfl_sync(0xffffffffu, mine.tiles, at);
        cur.w.chunks = __shfl_sync(0xffffffffu, mine.chunks, at);
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    const uint32_t per = kItemCost + cur.w.chunks, seg = (u0 - before) / per;
    cur.h = static_cast<int>(seg / cur.w.tiles);
    cur.tile = static_cast<int>(seg % cur.w.tiles);
    cur.left = shares.begin(me + 1) - u0;
    cur.base = before + seg * per;
    enter(cur, static_cast<int>(u0 - cur.base));
    if (cur.lo >= cur.hi && !advance<kRows>(cur, a, G)) return;
  }

  if (warp == kWarps) {
    // ---- the copies: lane w keeps warp w's ring filled, on its own way through the segments. The
    // lanes poll together (a lane that blocked would hold up the others), and each has loaded its
    // next unit's page numbers long before it needs them.
    if (lane >= kWarps) return;
    constexpr uint32_t kLanes = (1u << kWarps) - 1u;
    const int shift = a.c.page_shift - 4;
    Cursor at = cur;
    int unit = at.lo + lane, records = 0, given = 0;
    int page[kUnitRecords] = {};
    bool more = true;
    auto look = [&]() {
      while (more && unit >= at.hi) {
        more = advance<kRows>(at, a, G);
        unit = at.lo + lane;
      }
      if (!more) return;
      records = min(kUnitRecords, (at.w.s.n + 15) / 16 - unit * kUnitRecords);
      const int32_t* table = a.c.table + static_cast<size_t>(at.b) * a.c.width;
#pragma unroll
      for (int j = 0; j < kUnitRecords; ++j)
        if (j < records) page[j] = table[(unit * kUnitRecords + j) >> shift];
    };
    look();
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    uint64_t since = 0;  // when polling began to no avail
    bool ok = true;
    while (__any_sync(kLanes, more)) {
      const int stage = lane * kStages + given % kStages;
      const bool free = more && (given < kStages ||
                                 mbar_test(&empty[stage], (given / kStages - 1) & 1u));
      if (free) {
        const uint8_t* src[kUnitRecords];
        uint32_t has = 0;
#pragma unroll
        for (int j = 0; j < kUnitRecords; ++j) {
          src[j] = j < records ? kv4_in_page(a.c, page[j], at.h, unit * kUnitRecords + j, R::kBytes)
                               : nullptr;
          if (src[j] != nullptr) has |= 1u << j;
        }
        uint8_t* dst = smem + stage * S::stage_bytes;
        stage_has[stage] = has;
        if (has != (1u << records) - 1u) {
          // a page out of range: V scales of NaN send the unit to the masked body (64 sequences of
          // 8192 with weights 132.8 us; 133.4 with a look at stage_has for every unit)
          for (int j = 0; j < records; ++j)
            for (int x = 0; !((has >> j) & 1u) && x < 16 * NG; ++x)
              reinterpret_cast<uint32_t*>(dst + j * R::kBytes + R::kVParams)[x] = 0xFFFFFFFFu;
          fence_proxy_async();  // before the copies that this place holds later
        }
        mbar_arrive_expect_tx(&full[stage], __popc(has) * R::kBytes);
        if (shift > 0 && has == kAllRecords) {
          bulk_load_once(dst, src[0], kUnitRecords * R::kBytes, &full[stage], policy);  // one page
        } else {
#pragma unroll
          for (int j = 0; j < kUnitRecords; ++j)
            if (src[j] != nullptr)
              bulk_load_once(dst + j * R::kBytes, src[j], R::kBytes, &full[stage], policy);
        }
        ++given;
        unit += kWarps;
        look();
      }
      if (__any_sync(kLanes, free)) {
        since = 0;
        continue;
      }
      const uint64_t now = global_timer_ns();
      if (since == 0) since = now;
      if (__any_sync(kLanes, *abort_flag != 0u || now - since > a.wait_limit_ns)) {
        ok = false;
        *abort_flag = 1u;
        if (lane == 0) atomicOr(a.c.status, kStatusTimeout);
        break;
      }
      __nanosleep(32);
    }
    if (!ok) {  // copies in flight land before the CTA exits
      volatile uint32_t no_abort = 0u;
      for (int i = max(0, given - kStages); i < given; ++i)
        mbar_wait_bounded(&full[lane * kStages + i % kStages], (i / kStages) & 1u, &no_abort,
                          a.c.status, a.wait_limit_ns);
    }
    return;
  }

  const int r = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * kStages * S::stage_bytes;
  const uint32_t q_s = smem_addr(smem) + S::q_off + lane * 16;
  float* sm_o = reinterpret_cast<float*>(smem + S::o_off);
  float2* sm_ml = reinterpret_cast<float2*>(smem + S::ml_off);
  float* sm_row = reinterpret_cast<float*>(smem + S::row_off);  // [NG + 1][row]
  // its sign, or a zero, goes into q: hidden logits are -inf times this
  const float scale2 = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * kLog2e;
  int used = 0;
  bool ok = true;
  for (;;) {
    const Kv4Seq seq = cur.w.s;
    const int row0 = cur.tile * kRows, rows = min(kRows, seq.m * G - row0);
    // ---- a warp an n8 tile brings the queries into FP16 fragments under a power of two a row
    if (warp < NT) {
      const int row = row0 + warp * 8 + (PACK ? r & 3 : r);
      const bool have = row - row0 < rows;
      const uint16_t* src = a.q + static_cast<int64_t>(seq.s0 + (have ? row / G : 0)) * a.q_stride +
                            (cur.h * G + (have ? row % G : 0)) * D + 8 * c;
      uint4 v[NB];
      uint32_t top = 0;  // largest magnitude of the row, BF16 bits
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        v[x] = make_uint4(0, 0, 0, 0);
        if (have) v[x] = __ldg(reinterpret_cast<const uint4*>(src + 32 * x));
      }
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^up brings the row's largest to [2^14, 2^15)
      const int ex = static_cast<int>(top >> 7);
      const int up = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -126), 126);
      const float f = a.scale < 0.f ? -pow2f(up) : a.scale > 0.f ? pow2f(up) : 0.f;
      const float f16 = f * 0.0625f;  // pairs 1 and 3 meet codes times 16
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const uint4 h = make_uint4(f16x2_bits(bf16_lo(v[x].x) * f, bf16_hi(v[x].x) * f),
                                   f16x2_bits(bf16_lo(v[x].y) * f16, bf16_hi(v[x].y) * f16),
                                   f16x2_bits(bf16_lo(v[x].z) * f, bf16_hi(v[x].z) * f),
                                   f16x2_bits(bf16_lo(v[x].w) * f16, bf16_hi(v[x].w) * f16));
        uint4* to = reinterpret_cast<uint4*>(smem + S::q_off + ((warp * NB + x) * 32 + lane) * 16);
        if constexpr (PACK) {
          const uint4 none = make_uint4(0, 0, 0, 0);
          to[0] = r < 4 ? h : none;
          to[NB * 32] = r < 4 ? none : h;
        } else {
          *to = h;
        }
        v[x] = h;
      }
      // sums of q over a group's dims, as codes 1 would give them: column n of the product
      constexpr uint32_t one = 0x00040004u, one16 = 0x00400040u;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float acc[4];
#pragma unroll
        for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x) {
          if (x == g * NB / NG)
            mma_f16_first(acc, one, one, one16, one16, v[x].x, v[x].y);
          else
            mma_f16_16816(acc, one, one, one16, one16, v[x].x, v[x].y);
          mma_f16_16816(acc, one, one, one16, one16, v[x].z, v[x].w);
        }
        if (r == 0) {
          sm_row[g * kRows + warp * 8 + 2 * c] = acc[0];
          sm_row[g * kRows + warp * 8 + 2 * c + 1] = acc[1];
        }
      }
      // products are codes' 2^22 too small, as the sums are
      if (c == 0)
        sm_row[NG * kRows + warp * 8 + r] = fmaxf(scale2 * 4194304.f * pow2f(-up), 1e-37f);
    }
    join_warps();
    float sq[NT][NG][2], unscale[NT][2];  // of rows 2c, 2c + 1
    float o[NT][NB][2][4], corr[NT][NG][2], mx[NT][2], sum[NT][2];
    int ev[NT][2];         // exponent field of the rows' largest products under the maximum
    float down[NT][2];     // 2^(kLift - ev)
    float cap = -1.f;      // V scales up to this may come under every row's 2^-ev
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = nt * 8 + 2 * c + i;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          sq[nt][g][i] = sm_row[g * kRows + row];
          corr[nt][g][i] = 0.f;
        }
        unscale[nt][i] = sm_row[NG * kRows + row];
        mx[nt][i] = -INFINITY;
        sum[nt][i] = 0.f;
        ev[nt][i] = kLeastEv;
        down[nt][i] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[nt][x][y][z] = 0.f;
    }
    // first key that some row of the tile does not see
    const int clear = rows > 0 ? seq.n - seq.m + row0 / G + 1 : 0;

    // Records of bits `has`; false, with nothing done, if the body without a mask met a unit that
    // does not have all of them.
    auto compute = [&](auto mask, uint32_t base, int key0, volatile uint32_t* stage_bits) {
      constexpr bool kMasked = decltype(mask)::value;
      const uint32_t has = kMasked ? *stage_bits : kAllRecords;
      // ---- logits. Set j holds record j's tokens (packed: the lane's record's)
      constexpr int kSets = PACK ? 1 : kUnitRecords;
      const int half = c >> 1;  // packed: this lane's record
      float s[kSets][NT][4];
      auto fold = [&](int j, int g, uint32_t p0, uint32_t p1, const float (&acc)[NT][4]) {
        const float s0 = bf16_lo(p0), s1 = bf16_lo(p1), m0 = bf16_hi(p0), m1 = bf16_hi(p1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float m = i < 2 ? m0 : m1, sum_q = sq[nt][g][i & 1];
            s[j][nt][i] = fmaf(i < 2 ? s0 : s1, acc[nt][i],
                               g == 0 ? m * sum_q : fmaf(m, sum_q, s[j][nt][i]));
          }
      };
      auto hide_and_keep = [&](int j) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = PACK ? 2 * (c & 1) + (i & 1) : nt * 8 + 2 * c + (i & 1);
            const int key = key0 + 16 * (PACK ? half : j) + r + (i >= 2 ? 8 : 0);
            // rounded before the maximum comes off: a logit of 2^28 and more would overflow P by
            // what an fma keeps of it beyond the maximum
            s[j][nt][i] = __fmul_rn(s[j][nt][i], unscale[nt][i & 1]);
            if constexpr (kMasked) {
              if (key > (row < rows ? seq.n - seq.m + (row0 + row) / G : -1) ||
                  !((has >> (PACK ? half : j)) & 1u))
                s[j][nt][i] = -INFINITY;
            }
            if constexpr (LOGITS) {
              if (row < rows && key < seq.n)
                ws.logits[((static_cast<size_t>(cur.b) * a.c.kv_heads + cur.h) * a.max_new * G +
                           row0 + row) * ws.row_len + key] = s[j][nt][i];
            }
          }
      };
      if constexpr (PACK) {
        uint32_t w0[kUnitRecords][NB], w1[kUnitRecords][NB];
#pragma unroll
        for (int j = 0; j < kUnitRecords; ++j) {
          load_words<NB>(base + j * R::kBytes + ((r * 4 + c) * NB) * 4, w0[j]);
          load_words<NB>(base + j * R::kBytes + (((r + 8) * 4 + c) * NB) * 4, w1[j]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t at = base + half * R::kBytes + R::kKParams + (16 * g + r) * 4;
          const uint32_t p0 = lds32(at), p1 = lds32(at + 32);
          float acc[NT][4];
#pragma unroll
          for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x)
#pragma unroll
            for (int j = 0; j < kUnitRecords; ++j) {
              uint32_t k0[4], k1[4];
              key_pairs(w0[j][x], k0);
              key_pairs(w1[j][x], k1);
              const uint4 q = lds128(q_s + (j * NB + x) * 512);
              if (x == g * NB / NG && j == 0)
                mma_f16_first(acc[0], k0[0], k1[0], k0[1], k1[1], q.x, q.y);
              else
                mma_f16_16816(acc[0], k0[0], k1[0], k0[1], k1[1], q.x, q.y);
              mma_f16_16816(acc[0], k0[2], k1[2], k0[3], k1[3], q.z, q.w);
            }
          fold(0, g, p0, p1, acc);
        }
        hide_and_keep(0);
      } else {
#pragma unroll
        for (int j = 0; j < kUnitRecords; ++j) {
          if (kMasked && !((has >> j) & 1u)) {
            hide_and_keep(j);
            continue;
          }
          const uint32_t rec = base + j * R::kBytes;
          uint32_t w0[NB], w1[NB];
          load_words<NB>(rec + ((r * 4 + c) * NB) * 4, w0);
          load_words<NB>(rec + (((r + 8) * 4 + c) * NB) * 4, w1);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const uint32_t p0 = lds32(rec + R::kKParams + (16 * g + r) * 4);
            const uint32_t p1 = lds32(rec + R::kKParams + (16 * g + r + 8) * 4);
            float acc[NT][4];
#pragma unroll
            for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x) {
              uint32_t k0[4], k1[4];
              key_pairs(w0[x], k0);
              key_pairs(w1[x], k1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint4 q = lds128(q_s + (nt * NB + x) * 512);
                if (x == g * NB / NG)
                  mma_f16_first(acc[nt], k0[0], k1[0], k0[1], k1[1], q.x, q.y);
                else
                  mma_f16_16816(acc[nt], k0[0], k1[0], k0[1], k1[1], q.x, q.y);
                mma_f16_16816(acc[nt], k0[2], k1[2], k0[3], k1[3], q.z, q.w);
              }
            }
            fold(j, g, p0, p1, acc);
          }
          hide_and_keep(j);
        }
      }
      // ---- running maximum, and the largest product's exponent under it. Both may lag: p times a
      // scale stays an FP16 number, and most units need neither the reductions over the warp nor a
      // rescale.
      constexpr int kScales = kUnitRecords * NG * 16;
      auto scale_bits = [&](int x) {
        return lds32(base + (x / (16 * NG)) * R::kBytes + R::kVParams + (x % (16 * NG)) * 4) &
               0xFFFFu;
      };
      bool fits = !kMasked;
      if constexpr (!kMasked) {
#pragma unroll
        for (int x = 0; x < kScales; x += 32)
          fits = fits && __uint_as_float(scale_bits(x + lane) << 16) <= cap;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
#pragma unroll
            for (int j = 1; j < kSets; ++j)
              v = fmaxf(v, fmaxf(s[j][nt][i], s[j][nt][i + 2]));
            fits = fits && v <= mx[nt][i] + kLag;
          }
      }
      if (kMasked || !__all_sync(0xffffffffu, fits)) {
        if (!kMasked && *stage_bits != kAllRecords) return false;
        float reach[kSets][2];  // largest V scale of the lane's tokens
#pragma unroll
        for (int j = 0; j < kSets; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t top = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const uint32_t z = lds32(base + (PACK ? half : j) * R::kBytes + R::kVParams +
                                       (16 * g + r + 8 * u) * 4) & 0xFFFFu;
              if (z < 0x7F80u) top = max(top, z);
            }
            reach[j][u] = __uint_as_float(top << 16);
          }
        int least = 255;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
#pragma unroll
            for (int j = 1; j < kSets; ++j)
              v = fmaxf(v, fmaxf(s[j][nt][i], s[j][nt][i + 2]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            if constexpr (PACK) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            const float now = fmaxf(mx[nt][i], v);
            uint32_t top = 0;  // largest product, fp32 bits
#pragma unroll
            for (int j = 0; j < kSets; ++j)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float x = s[j][nt][i + 2 * u];
                if (kMasked && x == -INFINITY) continue;
                top = max(top, __float_as_uint(ex2(x - now) * reach[j][u]));
              }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float alpha = now == -INFINITY ? 1.f : ex2(mx[nt][i] - now);
            // the largest product so far is alpha times what it was
            const int before = ev[nt][i] + static_cast<int>(__float_as_uint(alpha) >> 23) - 127;
            const int ev_now = max(max(before, static_cast<int>(top >> 23)), kLeastEv);
            const float beta = alpha * ex2(static_cast<float>(ev[nt][i] - ev_now));
            mx[nt][i] = now;
            ev[nt][i] = ev_now;
            down[nt][i] = pow2f(127 + kLift - min(ev_now, 250));
            least = min(least, ev_now);
            sum[nt][i] *= alpha;
#pragma unroll
            for (int g = 0; g < NG; ++g) corr[nt][g][i] *= alpha;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                o[nt][x][y][i] *= beta;
                o[nt][x][y][i + 2] *= beta;
              }
          }
        least = __reduce_min_sync(0xffffffffu, least);
        cap = pow2f(min(least + kScaleLag - 127, 127));
      }
      // ---- P V
      auto probabilities = [&](int j, float (&p)[NT][4], float (&pd)[NT][4]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float m = mx[nt][i & 1];
            p[nt][i] = ex2(s[j][nt][i] - (kMasked && m == -INFINITY ? 0.f : m));
            sum[nt][i & 1] += p[nt][i];
            pd[nt][i] = p[nt][i] * down[nt][i & 1];
          }
      };
      // P of set j times group g's scales (parameters p0, p1), as the products' second operand
      auto scaled = [&](int j, int g, uint32_t p0, uint32_t p1, const float (&p)[NT][4],
                        const float (&pd)[NT][4], uint32_t (&b0)[NT], uint32_t (&b1)[NT]) {
        const float s0 = bf16_lo(p0), s1 = bf16_lo(p1), m0 = bf16_hi(p0), m1 = bf16_hi(p1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = pd[nt][i] * (i < 2 ? s0 : s1);
            // a hidden token's parameters may hold anything, NaN included
            if (kMasked && s[j][nt][i] == -INFINITY)
              x[i] = 0.f;
            else
              corr[nt][g][i & 1] = fmaf(p[nt][i], i < 2 ? m0 : m1, corr[nt][g][i & 1]);
          }
          b0[nt] = movmatrix_trans(f16x2_bits(x[0], x[1]));
          b1[nt] = movmatrix_trans(f16x2_bits(x[2], x[3]));
        }
      };
      if constexpr (PACK) {
        float p[NT][4], pd[NT][4];
        probabilities(0, p, pd);
        uint32_t w0[kUnitRecords][NB], w1[kUnitRecords][NB];
#pragma unroll
        for (int j = 0; j < kUnitRecords; ++j) {
          load_words<NB>(base + j * R::kBytes + R::kV + ((c * 8 + r) * NB) * 4, w0[j]);
          load_words<NB>(base + j * R::kBytes + R::kV + (((c + 4) * 8 + r) * NB) * 4, w1[j]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t at = base + half * R::kBytes + R::kVParams + (16 * g + r) * 4;
          uint32_t b0[NT], b1[NT];
          scaled(0, g, lds32(at), lds32(at + 32), p, pd, b0, b1);
#pragma unroll
          for (int j = 0; j < kUnitRecords; ++j) {
            // a lane holds a column: the other record's are no part of this one's product
            const bool on = (r >= 4) == (j == 1);
            const uint32_t c0 = on ? b0[0] : 0u, c1 = on ? b1[0] : 0u;
#pragma unroll
            for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x) {
              uint32_t v0[4], v1[4];
              value_pairs(w0[j][x], v0);
              value_pairs(w1[j][x], v1);
              mma_f16_16816(o[0][x][0], v0[0], v0[1], v1[0], v1[1], c0, c1);
              mma_f16_16816(o[0][x][1], v0[2], v0[3], v1[2], v1[3], c0, c1);
            }
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kUnitRecords; ++j) {
          if (kMasked && !((has >> j) & 1u)) continue;
          const uint32_t rec = base + j * R::kBytes;
          uint32_t w0[NB], w1[NB];
          load_words<NB>(rec + R::kV + ((c * 8 + r) * NB) * 4, w0);
          load_words<NB>(rec + R::kV + (((c + 4) * 8 + r) * NB) * 4, w1);
          float p[NT][4], pd[NT][4];
          probabilities(j, p, pd);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const uint32_t at = rec + R::kVParams + (16 * g + r) * 4;
            uint32_t b0[NT], b1[NT];
            scaled(j, g, lds32(at), lds32(at + 32), p, pd, b0, b1);
#pragma unroll
            for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x) {
              uint32_t v0[4], v1[4];
              value_pairs(w0[x], v0);
              value_pairs(w1[x], v1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(o[nt][x][0], v0[0], v0[1], v1[0], v1[1], b0[nt], b1[nt]);
                mma_f16_16816(o[nt][x][1], v0[2], v0[3], v1[2], v1[3], b0[nt], b1[nt]);
              }
            }
          }
        }
      }
      return true;
    };

#pragma unroll 1
    for (int unit = cur.lo + warp; unit < cur.hi; unit += kWarps) {
      const int stage = used % kStages;
      if (ok)
        ok = mbar_wait_bounded(&full[warp * kStages + stage], (used / kStages) & 1u, abort_flag,
                               a.c.status, a.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      ++used;
      if (!ok) continue;
      const uint32_t base = ring + stage * S::stage_bytes;
      const int key0 = unit * kUnit;
      volatile uint32_t* bits = &stage_has[warp * kStages + stage];
      // two bodies: the one that every unit but a sequence's last takes has no branches
      if (key0 + kUnit > clear || !compute(std::false_type(), base, key0, bits))
        compute(std::true_type(), base, key0, bits);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[warp * kStages + stage]);
    }

    // ---- join the warps: every warp under the rows' common maximum, the upper half's
    // accumulators onto the lower half's, then those (packed: all at once).
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = sum[nt][i];
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1)
            corr[nt][g][i] += __shfl_xor_sync(0xffffffffu, corr[nt][g][i], d);
        if (r == 0) sm_ml[warp * kRows + nt * 8 + 2 * c + i] = make_float2(mx[nt][i], l);
      }
    join_warps();
    // an accumulator's dims 32 x + 4 r .. of column 2 c + i, under the rows' common maximum
    auto share_of = [&](int nt, int i, float4 (&v)[NB]) {
      const int row = nt * 8 + 2 * c + i;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_ml[w * kRows + row].x);
      const float w = mx[nt][i] == -INFINITY ? 0.f : ex2(mx[nt][i] - m);
      // sums of codes' 2^-24, 2^-20, 2^-22, 2^-18 by dims, under 2^(kLift - ev)
      const float f = pow2f(min(ev[nt][i], 250) - 127), two = pow2f(24 - kLift);
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const float k = corr[nt][x / (NB / NG)][i];
        v[x] = make_float4(fmaf(o[nt][x][0][i] * two, f, k),
                           fmaf(o[nt][x][0][i + 2] * (two * 0.0625f), f, k),
                           fmaf(o[nt][x][1][i] * (two * 0.25f), f, k),
                           fmaf(o[nt][x][1][i + 2] * (two * 0.015625f), f, k));
        v[x] = w == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : make_float4(v[x].x * w, v[x].y * w, v[x].z * w, v[x].w * w);
      }
    };
    if constexpr (PACK) {
      // a row's two columns are two lanes' (c and c ^ 2): each sums one of the pair's rows
      float4 keep[NB], give[NB];
      share_of(0, 0, keep);
      share_of(0, 1, give);
      const int row = 2 * (c & 1) + (c >> 1);
      auto sum_of = [&](float a, float b) {
        const float mine = (c >> 1) ? b : a, other = (c >> 1) ? a : b;
        return mine + __shfl_xor_sync(0xffffffffu, other, 2);
      };
#pragma unroll
      for (int x = 0; x < NB; ++x)
        *reinterpret_cast<float4*>(sm_o + (warp * 4 + row) * D + 32 * x + 4 * r) = make_float4(
            sum_of(keep[x].x, give[x].x), sum_of(keep[x].y, give[x].y),
            sum_of(keep[x].z, give[x].z), sum_of(keep[x].w, give[x].w));
      join_warps();
    } else {
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        if ((warp < kLower) == (pass == 1)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float4 v[NB];
              share_of(nt, i, v);
#pragma unroll
              for (int x = 0; x < NB; ++x) {
                float4* at = reinterpret_cast<float4*>(
                    sm_o + ((warp % kLower) * kRows + nt * 8 + 2 * c + i) * D + 32 * x + 4 * r);
                if (pass == 1 && warp + kLower < kWarps) {
                  const float4 t = *at;
                  v[x] = make_float4(v[x].x + t.x, v[x].y + t.y, v[x].z + t.z, v[x].w + t.w);
                }
                *at = v[x];
              }
            }
        }
        join_warps();
      }
    }
    const bool whole = cur.lo == 0 && cur.hi == cur.w.chunks;
    auto part_of = [&](uint32_t cta, bool first) {
      return ws.parts + static_cast<size_t>(2 * cta + (first ? 1 : 0)) * S::part_floats;
    };
    float* part = part_of(me, cur.lo == 0);
    // (value, max, sum) of a row's dims 4 e .. 4 e + 3 -> output
    auto store = [&](int row, int e, float4 v, float m, float l) {
      const int rr = row0 + row;
      const int64_t at = static_cast<int64_t>(seq.s0 + rr / G) * a.heads + cur.h * G + rr % G;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      uint2 w = make_uint2(bf16x2_bits(v.x * inv, v.y * inv), bf16x2_bits(v.z * inv, v.w * inv));
      if (l == 0.f) w = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(a.out + at * D + 4 * e) = w;
      if (e == 0) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (a.lse != nullptr) a.lse[at] = lse2 * kLn2;
        if constexpr (LOGITS) ws.lse2[at] = lse2;
      }
    };
    for (int x = threadIdx.x; x < rows * (D / 4); x += kWarps * 32) {
      const int row = x / (D / 4), e = x % (D / 4);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_ml[w * kRows + row].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = sm_ml[w * kRows + row];
        if (ml.x != -INFINITY)
          l = fmaf(PACK ? ml.y + sm_ml[w * kRows + row + 4].y : ml.y, ex2(ml.x - m), l);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < (PACK ? kWarps : kLower); ++w) {
        const float4 t =
            *reinterpret_cast<const float4*>(sm_o + (w * (PACK ? 4 : kRows) + row) * D + 4 * e);
        v = make_float4(v.x + t.x, v.y + t.y, v.z + t.z, v.w + t.w);
      }
      if (whole) {
        store(row, e, v, m, l);
      } else {
        __stcg(reinterpret_cast<float4*>(part + row * D + 4 * e), v);
        if (e == 0)
          __stcg(reinterpret_cast<float2*>(part + kRows * D + 2 * row), make_float2(m, l));
      }
    }
    if (!whole) {
      // CTAs i0 .. i1 share the item; the one that arrives last joins their parts in order.
      const uint32_t first_unit = cur.base + kItemCost;
      const uint32_t i0 = shares.of(first_unit), i1 = shares.of(first_unit + cur.w.chunks - 1);
      join_warps();
      if (threadIdx.x == 0) {
        __threadfence();  // the CTA's writes, which the barrier has ordered before this
        uint32_t* cnt = ws.counters + i0;
        const bool last = atomicAdd(cnt, 1u) == i1 - i0;
        if (last) *cnt = 0u;
        __threadfence();
        *arrived = last ? 1u : 0u;
      }
      join_warps();
      if (*arrived) {
        // D / 4 lanes take a row, 4 dims each; together they read the parts' (max, sum), a lane
        // a part, and then each its dims of the parts, eight at a time.
        constexpr int kLanes = D / 4;
        const int e = threadIdx.x % kLanes;
        const int count = static_cast<int>(i1 - i0) + 1;
        for (int row = threadIdx.x / kLanes; row < (rows + 1) / 2 * 2;
             row += kWarps * 32 / kLanes) {
          auto ml_of = [&](int i) {
            return row < rows && i < count
                       ? __ldcg(reinterpret_cast<const float2*>(part_of(i0 + i, i == 0) +
                                                                kRows * D + 2 * row))
                       : make_float2(-INFINITY, 0.f);
          };
          float m = -INFINITY;
          for (int i = e; i < (count + kLanes - 1) / kLanes * kLanes; i += kLanes)
            m = fmaxf(m, ml_of(i).x);
#pragma unroll
          for (int o2 = kLanes / 2; o2 > 0; o2 >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o2));
          float l = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int base = 0; base < count; base += kLanes) {
            const float2 ml = ml_of(base + e);
            const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
            const float wl = w * ml.y;
            for (int j = 0; j < min(kLanes, count - base); j += 8) {
              float4 t[8];
#pragma unroll
              for (int x = 0; x < 8; ++x)
                t[x] = row < rows && base + j + x < count
                           ? __ldcg(reinterpret_cast<const float4*>(
                                 part_of(i0 + base + j + x, base + j + x == 0) + row * D + 4 * e))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float f = __shfl_sync(0xffffffffu, w, j + x, kLanes);
                l += __shfl_sync(0xffffffffu, wl, j + x, kLanes);
                if (f != 0.f) {
                  v.x = fmaf(t[x].x, f, v.x), v.y = fmaf(t[x].y, f, v.y);
                  v.z = fmaf(t[x].z, f, v.z), v.w = fmaf(t[x].w, f, v.w);
                }
              }
            }
          }
          if (row < rows) store(row, e, v, m, l);
        }
      }
    }
    if (!advance<kRows>(cur, a, G)) break;
    join_warps();  // the join's reads of shared memory before the next segment's writes
  }
}

// weights_out[b, h, j] = weights[b, h, j] + sum over rows of exp2(logit - lse2), in row order.
// A thread takes four tokens 256 apart, four rows of each at a time: sixteen loads on their way.
constexpr int kFewRows = 96;  // rows a key/value head has at most on this path
__global__ void __launch_bounds__(256) kv4_weights_kernel(const Kv4AttentionArgs a,
                                                          const Workspace ws) {
  __shared__ float lse[kFewRows];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y, G = a.heads / a.c.kv_heads;
  const Kv4Seq s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
  const int key0 = blockIdx.x * 1024 + threadIdx.x;
  if (blockIdx.x * 1024 >= s.n) return;
  const int rows = s.m * G;
  if (threadIdx.x < kFewRows) {
    float v = INFINITY;
    if (threadIdx.x < rows)
      v = ws.lse2[static_cast<int64_t>(s.s0 + threadIdx.x / G) * a.heads + h * G + threadIdx.x % G];
    lse[threadIdx.x] = v == -INFINITY ? INFINITY : v;  // such a row adds nothing
  }
  __syncthreads();
  const size_t bh = static_cast<size_t>(b) * a.c.kv_heads + h;
  const float* x = ws.logits + bh * a.max_new * G * ws.row_len + key0;
  const size_t at = bh * a.weights_stride + key0;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (a.weights != nullptr && key0 + 256 * t < s.n) w[t] = a.weights[at + 256 * t];
  for (int row = 0; row < rows; row += 4) {
    float v[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        v[r][t] = row + r < rows && key0 + 256 * t < s.n
                      ? x[static_cast<size_t>(row + r) * ws.row_len + 256 * t]
                      : -INFINITY;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] += ex2(v[r][t] - lse[row + r]);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (key0 + 256 * t < s.n) a.weights_out[at + 256 * t] = w[t] + acc[t];
}

// n8 tiles of a row tile. More than two are slower than several row tiles of two: head size 64,
// 36 rows in three tiles 12.9 us (one sequence of 2048), 32 rows in one of four 18.0 us.
int row_blocks(int max_new, int G) { return max_new * G <= 8 ? 1 : 2; }

struct Layout {
  size_t lse2, logits, parts, total;
  int row_len;
};
int grid_limit(int d, int nt) {  // a counter a CTA
  const int n = ctas_per_sm(d, nt) * device_sm_count(), most = kKv4CounterBytes / 4;
  return n < most ? n : most;
}

Layout layout(int batch, int tokens, int max_new, int max_len, int heads, int kv_heads, int D,
              bool weights) {
  Layout l;
  const int G = heads / kv_heads, nt = row_blocks(max_new, G);
  l.row_len = (max_len + 3) / 4 * 4;
  size_t at = kKv4CounterBytes;
  l.parts = at;
  at += round256(static_cast<size_t>(2) * grid_limit(D, nt) * nt * 8 * (D + 2) * 4);
  l.lse2 = at;
  if (weights) at += round256(static_cast<size_t>(tokens) * heads * 4);
  l.logits = at;
  if (weights)
    at += round256(static_cast<size_t>(batch) * heads * max_new * l.row_len * 4);
  l.total = at;
  return l;
}

template <int D, int NG, int NT, bool PACK>
cudaError_t run(const Kv4AttentionArgs& a, cudaStream_t stream) {
  using S = Shape<D, NG, NT, PACK>;
  const Layout l = layout(a.c.batch, a.tokens, a.max_new, a.max_len, a.heads, a.c.kv_heads, D,
                          a.weights_out != nullptr);
  Workspace ws;
  ws.counters = reinterpret_cast<uint32_t*>(a.workspace);
  ws.lse2 = reinterpret_cast<float*>(a.workspace + l.lse2);
  ws.logits = reinterpret_cast<float*>(a.workspace + l.logits);
  ws.parts = reinterpret_cast<float*>(a.workspace + l.parts);
  ws.row_len = l.row_len;
  auto kern = a.weights_out != nullptr ? kv4_attention_kernel<D, NG, NT, PACK, true>
                                       : kv4_attention_kernel<D, NG, NT, PACK, false>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), S::total);
  if (e != cudaSuccess) return e;
  const int G = a.heads / a.c.kv_heads;
  const int64_t tiles = (static_cast<int64_t>(a.max_new) * G + S::kRows - 1) / S::kRows;
  const int64_t units = static_cast<int64_t>(a.c.batch) * a.c.kv_heads * tiles *
                        (kItemCost + (a.max_len + kUnit - 1) / kUnit);
  if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int64_t want = (units + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(want < grid_limit(D, NT) ? want : grid_limit(D, NT));
  e = launch_with_pdl(kern, dim3(grid), dim3((kWarps + 1) * 32), S::total, stream, a, ws);
  if (e != cudaSuccess || a.weights_out == nullptr) return e;
  return launch_with_pdl(kv4_weights_kernel,
                         dim3((a.max_len + 1023) / 1024, a.c.kv_heads, a.c.batch), dim3(256), 0,
                         stream, a, ws);
}

template <int D, int NG>
cudaError_t by_rows(const Kv4AttentionArgs& a, cudaStream_t stream) {
  const int G = a.heads / a.c.kv_heads;
  if (row_blocks(a.max_new, G) == 2) return run<D, NG, 2, false>(a, stream);
  return a.max_new * G <= 4 ? run<D, NG, 1, true>(a, stream) : run<D, NG, 1, false>(a, stream);
}

// Above kFewRows the prompts' path takes over. It widens the whole cache to FP16 tiles first and
// pads the rows to 128; here every 16 rows read the cache's codes again. 32 query heads on 8, us at
// 80 and 96 rows here / 100 and 128 there: 94, 111 / 105, 102 for 16 sequences of 2048, 226, 267 /
// 307, 298 for 16 of 8192, 42, 47 / 79, 78 for one of 16384. So the border is a compromise: for
// many short sequences it lies a little late, for one long one early, and there the next row costs
// 30 us.
bool is_prompt(int max_new, int heads, int kv_heads) {
  return static_cast<int64_t>(max_new) * (heads / kv_heads) > kFewRows;
}

}  // namespace

size_t kv4_attention_workspace(int batch, int tokens, int max_new, int max_len, int heads,
                               int kv_heads, int head_dim, int group, bool weights) {
  if (is_prompt(max_new, heads, kv_heads))
    return kv4_prompt_workspace(batch, tokens, max_new, max_len, heads, kv_heads, head_dim,
                                weights);
  return layout(batch, tokens, max_new, max_len, heads, kv_heads, head_dim, weights).total;
}

cudaError_t launch_kv4_attention(const Kv4AttentionArgs& a, int head_dim, int group,
                                 cudaStream_t stream) {
  if (is_prompt(a.max_new, a.heads, a.c.kv_heads))
    return launch_kv4_prompt(a, head_dim, group, stream);
  if (head_dim == 128)
    return group == 128 ? by_rows<128, 1>(a, stream)
           : group == 64 ? by_rows<128, 2>(a, stream) : by_rows<128, 4>(a, stream);
  return group == 64 ? by_rows<64, 1>(a, stream) : by_rows<64, 2>(a, stream);
}

}  // namespace w4k
