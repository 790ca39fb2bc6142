// Attention of a few new tokens over the 4-bit key/value cache.
//
//   s_ij = scale q_i . k_hat_j (j <= n - m + i),  p = softmax_j(s),  out_i = sum_j p_ij v_hat_j
//
// Rows are the (new token, query head) pairs that share a key/value head, 8 NT of them a tile.
// With c the code less 8 (c - 8 and c are both exact small numbers), s the scale and m the minimum
// plus 8 s, of a dim's group g,
//   q . k_hat_j = sum_g s_jg (sum_{d in g} q_d c_jd) + m_jg (sum_{d in g} q_d)
//   sum_j p_j v_hat_jd = sum_j (p_j s_jg) c_jd + sum_j p_j m_jg
// so the codes go to the tensor pipe as they are, as FP16 pairs (one LOP3 and one HFMA2 a pair),
// and the scales touch one number a token and group. The codes are centred because the MMA
// truncates its sums: left as 1024 + c or 128 + c the offset's own sum, hundreds of times the
// result over a long cache, took 1.2 % of it (131072 tokens). q is FP16 under a power of two a
// row, exact down to 2^-31 of the row's largest; p s is rounded to FP16 under the largest scale's
// power of two that the row has met (relative 2^-12; BF16's 2^-9 was twice the output's own
// rounding error). Sums, maxima and the softmax's statistics are fp32.
//
// What bounds it: the cache is read once (D + 8 D / group bytes a token and head), at 4 heads a
// key/value head about 8 operations a byte, so the aim is the memory's rate.
//
// Work split. A unit is 64 tokens of one (sequence, head, row tile); the units of all sequences
// in order are cut into equal ranges, one a CTA, from the lengths on the device: ragged batches
// and one long sequence use the whole GPU alike, and a bound on the length costs nothing. Within
// a range the CTA's warps take units in turn, each with its own ring of bulk copies and no
// barrier but at the end of a segment (the part of one sequence, head and tile in the range),
// where they join (max, sum, accumulator) through shared memory. A segment that another CTA
// shares goes to the workspace in fp32, and the CTA that arrives last joins the parts in order.
#include "kv4_common.cuh"
#include "kv4_prompt.h"

namespace w4k {
namespace {

constexpr int kWarps = 4;
constexpr int kUnit = 64;  // tokens
constexpr int kUnitRecords = kUnit / 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// FP16 pairs (q - 8, q' - 8) of nibbles i and i + 4, i = 0..3.
__device__ __forceinline__ void centred_pairs(uint32_t w, uint32_t (&p)[4]) {
  code_pairs_f16(w, p);  // 1024 + q (even i) and 1024 + 16 q (odd i)
  const __half2 one = __float2half2_rn(1.f), off = __float2half2_rn(-1032.f);
  const __half2 frac = __float2half2_rn(0.0625f), off16 = __float2half2_rn(-72.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 x = *reinterpret_cast<__half2*>(&p[i]);
    x = i % 2 == 0 ? __hfma2(x, one, off) : __hfma2(x, frac, off16);
    p[i] = *reinterpret_cast<uint32_t*>(&x);
  }
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

struct Workspace {
  uint32_t* counters;  // one a segment, zero between calls
  float* lse2;         // [tokens, heads], base 2
  float* logits;       // [batch, kv_heads, max_new G, row_len], base 2 (weights only)
  float* parts;        // [2 grid] x (8 NT rows x D + 16 NT)
  int row_len;
};

// The units of sequence b: sequences without new tokens have none, an empty one has one a tile
// (its rows are still to be written).
struct Work {
  Kv4Seq s;
  int tiles, chunks;
};
template <int ROWS>
__device__ __forceinline__ Work work_of(const Kv4AttentionArgs& a, int group, int b) {
  Work w;
  w.s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
  w.tiles = (w.s.m * group + ROWS - 1) / ROWS;
  w.chunks = max(1, (w.s.n + kUnit - 1) / kUnit);
  return w;
}

// Position in the list of units. A warp walks units w, w + kWarps, ... of each segment.
struct Cursor {
  int b, h, tile;      // segment
  Work w;
  int lo, hi;          // the segment's units in this CTA's range
  int64_t left;        // units of the range after this segment's
};

template <int ROWS>
__device__ __forceinline__ void enter(Cursor& c, const Kv4AttentionArgs& a, int first) {
  c.lo = first;
  c.hi = static_cast<int>(min(static_cast<int64_t>(c.w.chunks), first + c.left));
  c.left -= c.hi - c.lo;
}

// Next segment of the range; false at its end.
template <int ROWS>
__device__ __forceinline__ bool advance(Cursor& c, const Kv4AttentionArgs& a, int group) {
  if (c.left <= 0) return false;
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
  enter<ROWS>(c, a, 0);
  return true;
}

template <int D, int NG, int NT, int STAGES>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr uint32_t stage_bytes = kUnitRecords * Kv4Record<D, NG>::kBytes;
  static constexpr uint32_t ring_bytes = kWarps * STAGES * stage_bytes;
  static constexpr uint32_t o_off = ring_bytes;                            // [warp][row][D]
  static constexpr uint32_t ml_off = o_off + kWarps * kRows * D * 4;       // [warp][row] (m, l)
  static constexpr uint32_t bar_off = ml_off + kWarps * kRows * 8;
  static constexpr uint32_t misc_off = bar_off + kWarps * STAGES * 8;
  static constexpr uint32_t total = misc_off + 16;
  static constexpr int part_floats = kRows * D + 2 * kRows;
};

template <int D, int NG, int NT, int STAGES, bool LOGITS>
__global__ void __launch_bounds__(kWarps * 32, 2)
    kv4_attention_kernel(const Kv4AttentionArgs a, const Workspace ws) {
  using R = Kv4Record<D, NG>;
  using S = Shape<D, NG, NT, STAGES>;
  constexpr int NB = R::kBlocks, kRows = S::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::bar_off);
  volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + S::misc_off);
  volatile uint32_t* arrived = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int G = a.heads / a.c.kv_heads;

  if (threadIdx.x < kWarps * STAGES) mbar_init(&bars[threadIdx.x], 1);
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  // This CTA's range of units.
  int64_t total = 0;
  for (int base = 0; base < a.c.batch; base += 32) {
    int64_t u = 0;
    if (base + lane < a.c.batch) {
      const Work w = work_of<kRows>(a, G, base + lane);
      u = static_cast<int64_t>(w.tiles) * w.chunks * a.c.kv_heads;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    total += u;
  }
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), (total + kWarps - 1) / kWarps);
  const int64_t me = blockIdx.x;
  if (me >= ctas) return;
  const int64_t u0 = total * me / ctas, u1 = total * (me + 1) / ctas;
  if (u0 >= u1) return;

  Cursor cur;
  int64_t seg_base = 0;  // first unit of the current segment
  {
    int64_t before = 0;
    int b = 0;
    for (;; ++b) {
      const Work w = work_of<kRows>(a, G, b);
      const int64_t u = static_cast<int64_t>(w.tiles) * w.chunks * a.c.kv_heads;
      if (u0 < before + u) {
        cur.w = w;
        break;
      }
      before += u;
    }
    const int64_t seg = (u0 - before) / cur.w.chunks;
    cur.b = b;
    cur.h = static_cast<int>(seg / cur.w.tiles);
    cur.tile = static_cast<int>(seg % cur.w.tiles);
    cur.left = u1 - u0;
    seg_base = before + seg * cur.w.chunks;
    enter<kRows>(cur, a, static_cast<int>(u0 - seg_base));
  }

  // Ring: this warp's units in order, STAGES - 1 ahead of the one it computes on.
  const uint32_t ring = smem_addr(smem) + warp * STAGES * S::stage_bytes;
  uint64_t* full = bars + warp * STAGES;
  Cursor pre = cur;
  int pre_unit = cur.lo + warp;
  bool pre_more = true;
  int filled = 0, used = 0;  // units loaded, units computed
  bool ok = true;
  auto fill = [&]() {
    while (pre_more && pre_unit >= pre.hi) {
      pre_more = advance<kRows>(pre, a, G);
      pre_unit = pre.lo + warp;
    }
    if (!pre_more || !ok) return;
    const int stage = filled % STAGES;
    const int records = min(kUnitRecords, (pre.w.s.n + 15) / 16 - pre_unit * kUnitRecords);
    // one copy a run of records within a page; lane i looks the run of record i up
    const int per_page = 1 << (a.c.page_shift - 4);
    const int run = min(per_page, kUnitRecords);
    const uint8_t* src = nullptr;
    if (lane < records && lane % run == 0)
      src = kv4_record(a.c, a.c.table, a.c.width, pre.b, pre.h, pre_unit * kUnitRecords + lane,
                       R::kBytes);
    const uint32_t bytes = src == nullptr ? 0u : min(run, records - lane) * R::kBytes;
    uint32_t sum = bytes;
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(&full[stage], sum);
    __syncwarp();
    if (src != nullptr)
      bulk_load(smem + (warp * STAGES + stage) * S::stage_bytes + lane * R::kBytes, src, bytes,
                &full[stage]);
    ++filled;
    pre_unit += kWarps;
  };
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) fill();

  const float scale2 = a.scale * kLog2e;
  for (;;) {
    // ---- one segment
    const Kv4Seq seq = cur.w.s;
    const int rows_all = seq.m * G, row0 = cur.tile * kRows;
    const int rows = min(kRows, rows_all - row0);
    uint32_t q[NT][NB][4];   // FP16 under the row's power of two
    float sq[NT][NG][2];     // sums of q over a group's dims, rows 2c, 2c + 1
    float unscale[NT][2];    // scale log2(e) / power of two of rows 2c, 2c + 1
    int last_key[NT][2];     // last visible key of rows 2c, 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 8 + r;
      const bool have = nt * 8 + r < rows;
      const uint16_t* src = a.q + static_cast<int64_t>(seq.s0 + (have ? row / G : 0)) * a.q_stride +
                            (cur.h * G + (have ? row % G : 0)) * D + 8 * c;
      uint32_t top = 0;  // largest magnitude of the row, BF16 bits
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (have) v = __ldg(reinterpret_cast<const uint4*>(src + 32 * s));
        q[nt][s][0] = v.x, q[nt][s][1] = v.y, q[nt][s][2] = v.z, q[nt][s][3] = v.w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = max(top, max(q[nt][s][i] & 0x7FFFu, (q[nt][s][i] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e brings the row's largest to [2^14, 2^15)
      const int ex = static_cast<int>(top >> 7);
      const int up = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -126), 126);
      const float f = pow2f(up);
#pragma unroll
      for (int s = 0; s < NB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[nt][s][i] = f16x2_bits(bf16_lo(q[nt][s][i]) * f, bf16_hi(q[nt][s][i]) * f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = nt * 8 + 2 * c + i;
        last_key[nt][i] = rr < rows ? seq.n - seq.m + (row0 + rr) / G : -1;
        unscale[nt][i] = scale2 * pow2f(-__shfl_sync(0xffffffffu, up, (2 * c + i) * 4));
      }
      constexpr uint32_t ones = 0x3C003C00u;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = g * NB / NG; s < (g + 1) * NB / NG; ++s) {
          mma_f16_16816(acc, ones, ones, ones, ones, q[nt][s][0], q[nt][s][1]);
          mma_f16_16816(acc, ones, ones, ones, ones, q[nt][s][2], q[nt][s][3]);
        }
        sq[nt][g][0] = acc[0];
        sq[nt][g][1] = acc[1];
      }
    }
    float o[NT][NB][2][4], corr[NT][NG][2], mx[NT][2], sum[NT][2];
    int ev[NT][2];  // exponent field of the largest V scale that rows 2c, 2c + 1 have met
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[nt][x][y][z] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[nt][i] = -INFINITY;
        sum[nt][i] = 0.f;
        ev[nt][i] = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g) corr[nt][g][i] = 0.f;
      }
    }
    // first key that some row of the tile does not see
    const int clear = rows > 0 ? seq.n - seq.m + row0 / G + 1 : 0;

#pragma unroll 1
    for (int unit = cur.lo + warp; unit < cur.hi; unit += kWarps) {
      fill();
      const int stage = used % STAGES;
      if (ok)
        ok = mbar_wait_bounded(&full[stage], (used / STAGES) & 1u, abort_flag, a.c.status,
                               a.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      ++used;
      if (!ok) continue;
      const uint32_t base = ring + stage * S::stage_bytes;
      const int key0 = unit * kUnit;
      const int records = min(kUnitRecords, (seq.n - key0 + 15) / 16);
      const bool masked = key0 + kUnit > clear;
      // ---- logits, base 2
      float s[kUnitRecords][NT][4];
#pragma unroll
      for (int j = 0; j < kUnitRecords; ++j) {
        if (j >= records) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][nt][i] = -INFINITY;
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
          const float s0 = bf16_lo(p0), s1 = bf16_lo(p1);
          const float m0 = fmaf(8.f, s0, bf16_hi(p0)), m1 = fmaf(8.f, s1, bf16_hi(p1));
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
#pragma unroll
          for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x) {
            uint32_t k0[4], k1[4];
            centred_pairs(w0[x], k0);
            centred_pairs(w1[x], k1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_16816(acc[nt], k0[0], k1[0], k0[1], k1[1], q[nt][x][0], q[nt][x][1]);
              mma_f16_16816(acc[nt], k0[2], k1[2], k0[3], k1[3], q[nt][x][2], q[nt][x][3]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float t = fmaf(i < 2 ? s0 : s1, acc[nt][i], (i < 2 ? m0 : m1) * sq[nt][g][i & 1]);
              s[j][nt][i] = g == 0 ? t : s[j][nt][i] + t;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j][nt][i] *= unscale[nt][i & 1];
        if (masked) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + 16 * j + r + (i >= 2 ? 8 : 0) > last_key[nt][i & 1])
                s[j][nt][i] = -INFINITY;
        }
        if constexpr (LOGITS) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = nt * 8 + 2 * c + (i & 1);
              const int key = key0 + 16 * j + r + (i >= 2 ? 8 : 0);
              if (rr < rows && key < seq.n)
                ws.logits[((static_cast<size_t>(cur.b) * a.c.kv_heads + cur.h) * a.max_new * G +
                           row0 + rr) * ws.row_len + key] = s[j][nt][i];
            }
        }
      }
      // ---- running maximum, and the largest V scale's exponent among the visible tokens
      int unit_ev[NT][2];
      if (!masked) {
        uint32_t top = 0;
#pragma unroll
        for (int x = lane; x < kUnitRecords * NG * 16; x += 32) {
          const uint32_t sc = lds32(base + (x / (16 * NG)) * R::kBytes + R::kVParams +
                                    (x % (16 * NG)) * 4) & 0xFFFFu;
          top = max(top, sc >= 0x7F80u ? 0u : sc);
        }
        top = __reduce_max_sync(0xffffffffu, top) >> 7;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) unit_ev[nt][0] = unit_ev[nt][1] = static_cast<int>(top);
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < kUnitRecords; ++j) {
              if (j >= records) continue;
#pragma unroll
              for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint32_t sc = lds32(base + j * R::kBytes + R::kVParams +
                                            (16 * g + r + 8 * half) * 4) & 0xFFFFu;
                  if (s[j][nt][i + 2 * half] != -INFINITY && sc < 0x7F80u) top = max(top, sc);
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
            unit_ev[nt][i] = static_cast<int>(top >> 7);
          }
      }
      bool grow = false;
      float alpha[NT][2], beta[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
#pragma unroll
          for (int j = 1; j < kUnitRecords; ++j)
            v = fmaxf(v, fmaxf(s[j][nt][i], s[j][nt][i + 2]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          const float now = fmaxf(mx[nt][i], v);
          const int ev_now = max(ev[nt][i], unit_ev[nt][i]);
          alpha[nt][i] = now == -INFINITY ? 1.f : exp2f(mx[nt][i] - now);
          beta[nt][i] = alpha[nt][i] * exp2f(static_cast<float>(ev[nt][i] - ev_now));
          grow |= now > mx[nt][i] || ev_now > ev[nt][i];
          mx[nt][i] = now;
          ev[nt][i] = ev_now;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f = alpha[nt][i];
            sum[nt][i] *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g) corr[nt][g][i] *= f;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                o[nt][x][y][i] *= beta[nt][i];
                o[nt][x][y][i + 2] *= beta[nt][i];
              }
          }
      }
      float down[NT][2];  // 2^-ev
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) down[nt][i] = pow2f(127 - min(ev[nt][i], 250));
      // ---- P V
#pragma unroll
      for (int j = 0; j < kUnitRecords; ++j) {
        if (j >= records) continue;
        const uint32_t rec = base + j * R::kBytes;
        uint32_t w0[NB], w1[NB];
        load_words<NB>(rec + R::kV + ((c * 8 + r) * NB) * 4, w0);
        load_words<NB>(rec + R::kV + (((c + 4) * 8 + r) * NB) * 4, w1);
        float p[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float m = mx[nt][i & 1];
            p[nt][i] = m == -INFINITY ? 0.f : exp2f(s[j][nt][i] - m);
            sum[nt][i & 1] += p[nt][i];
          }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t p0 = lds32(rec + R::kVParams + (16 * g + r) * 4);
          const uint32_t p1 = lds32(rec + R::kVParams + (16 * g + r + 8) * 4);
          const float s0 = bf16_lo(p0), s1 = bf16_lo(p1);
          const float m0 = fmaf(8.f, s0, bf16_hi(p0)), m1 = fmaf(8.f, s1, bf16_hi(p1));
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = p[nt][i] * ((i < 2 ? s0 : s1) * down[nt][i & 1]);
              y[i] = p[nt][i] * (i < 2 ? m0 : m1);
            }
            if (masked) {  // a hidden token's parameters may hold anything, NaN included
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (s[j][nt][i] == -INFINITY) x[i] = y[i] = 0.f;
            }
            corr[nt][g][0] += y[0] + y[2];
            corr[nt][g][1] += y[1] + y[3];
            b0[nt] = movmatrix_trans(f16x2_bits(x[0], x[1]));
            b1[nt] = movmatrix_trans(f16x2_bits(x[2], x[3]));
          }
#pragma unroll
          for (int x = g * NB / NG; x < (g + 1) * NB / NG; ++x) {
            uint32_t v0[4], v1[4];
            centred_pairs(w0[x], v0);
            centred_pairs(w1[x], v1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_16816(o[nt][x][0], v0[0], v0[1], v1[0], v1[1], b0[nt], b1[nt]);
              mma_f16_16816(o[nt][x][1], v0[2], v0[3], v1[2], v1[3], b0[nt], b1[nt]);
            }
          }
        }
      }
      __syncwarp();  // every lane is done with the stage before it is filled again
    }

    // ---- join the warps
    float* sm_o = reinterpret_cast<float*>(smem + S::o_off);
    float2* sm_ml = reinterpret_cast<float2*>(smem + S::ml_off);
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
        const int row = nt * 8 + 2 * c + i;
        if (r == 0) sm_ml[warp * kRows + row] = make_float2(mx[nt][i], l);
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          const float k = corr[nt][x / (NB / NG)][i];
          const float f = pow2f(min(ev[nt][i], 250) - 127);
          *reinterpret_cast<float4*>(sm_o + (warp * kRows + row) * D + 32 * x + 4 * r) =
              make_float4(fmaf(o[nt][x][0][i], f, k), fmaf(o[nt][x][0][i + 2], f, k),
                          fmaf(o[nt][x][1][i], f, k), fmaf(o[nt][x][1][i + 2], f, k));
        }
      }
    __syncthreads();
    const bool whole = cur.lo == 0 && cur.hi == cur.w.chunks;
    float* part = ws.parts + (2 * me + (cur.lo == 0 ? 1 : 0)) * S::part_floats;
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
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_ml[w * kRows + row].x);
      float l = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = sm_ml[w * kRows + row];
        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
        const float4 t =
            *reinterpret_cast<const float4*>(sm_o + (w * kRows + row) * D + 4 * e);
        if (f != 0.f) {
          l = fmaf(ml.y, f, l);
          v.x = fmaf(t.x, f, v.x), v.y = fmaf(t.y, f, v.y);
          v.z = fmaf(t.z, f, v.z), v.w = fmaf(t.w, f, v.w);
        }
      }
      if (whole) {
        store(row, e, v, m, l);
      } else {
        __stcg(reinterpret_cast<float4*>(part + row * D + 4 * e), v);
        if (e == 0) __stcg(reinterpret_cast<float2*>(part + kRows * D + 2 * row), make_float2(m, l));
      }
    }
    if (!whole) {
      // CTAs i0 .. i1 share the segment; the one that arrives last joins their parts in order.
      const int64_t i0 = ((seg_base + 1) * ctas - 1) / total;
      const int64_t i1 = ((seg_base + cur.w.chunks) * ctas - 1) / total;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t* cnt = ws.counters + (static_cast<size_t>(cur.b) * a.c.kv_heads + cur.h) *
                                          ((a.max_new * G + kRows - 1) / kRows) + cur.tile;
        const uint32_t n = atomicAdd(cnt, 1u);
        const bool last = n == static_cast<uint32_t>(i1 - i0);
        if (last) *cnt = 0u;
        *arrived = last ? 1u : 0u;
      }
      __syncthreads();
      if (*arrived) {
        __threadfence();
        for (int x = threadIdx.x; x < rows * (D / 4); x += kWarps * 32) {
          const int row = x / (D / 4), e = x % (D / 4);
          float m = -INFINITY;
          for (int64_t i = i0; i <= i1; ++i)
            m = fmaxf(m, __ldcg(ws.parts + (2 * i + (i == i0 ? 1 : 0)) * S::part_floats +
                                kRows * D + 2 * row));
          float l = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int64_t i = i0; i <= i1; ++i) {
            const float* src = ws.parts + (2 * i + (i == i0 ? 1 : 0)) * S::part_floats;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(src + kRows * D + 2 * row));
            const float4 t = __ldcg(reinterpret_cast<const float4*>(src + row * D + 4 * e));
            if (ml.x == -INFINITY) continue;
            const float f = exp2f(ml.x - m);
            l = fmaf(ml.y, f, l);
            v.x = fmaf(t.x, f, v.x), v.y = fmaf(t.y, f, v.y);
            v.z = fmaf(t.z, f, v.z), v.w = fmaf(t.w, f, v.w);
          }
          store(row, e, v, m, l);
        }
      }
    }
    seg_base += cur.w.chunks;
    if (!advance<kRows>(cur, a, G)) break;
    __syncthreads();  // the join's reads of shared memory before the next segment's writes
  }
  // A warp that gave up lets its copies in flight land before the CTA exits.
  if (!ok) {
    volatile uint32_t no_abort = 0u;
    for (int i = max(0, filled - STAGES); i < filled; ++i)
      mbar_wait_bounded(&full[i % STAGES], (i / STAGES) & 1u, &no_abort, a.c.status,
                        a.wait_limit_ns);
  }
}

// weights_out[b, h, j] = weights[b, h, j] + sum over rows of exp2(logit - lse2), in row order.
__global__ void __launch_bounds__(256) kv4_weights_kernel(const Kv4AttentionArgs a,
                                                          const Workspace ws) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y, G = a.heads / a.c.kv_heads;
  const Kv4Seq s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
  const int key = blockIdx.x * 256 + threadIdx.x;
  if (key >= s.n) return;
  const float* x = ws.logits + (static_cast<size_t>(b) * a.c.kv_heads + h) * a.max_new * G *
                                   ws.row_len + key;
  const size_t at = (static_cast<size_t>(b) * a.c.kv_heads + h) * a.weights_stride + key;
  float acc = 0.f;
  for (int row = 0; row < s.m * G; ++row) {
    const float l = ws.lse2[static_cast<int64_t>(s.s0 + row / G) * a.heads + h * G + row % G];
    if (l != -INFINITY) acc += exp2f(x[static_cast<size_t>(row) * ws.row_len] - l);
  }
  a.weights_out[at] = (a.weights != nullptr ? a.weights[at] : 0.f) + acc;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kMaxTiles = 2;  // n8 tiles a row tile has at most

struct Layout {
  size_t counters, lse2, logits, parts, total;
  int row_len;
};
int grid_limit() { return 2 * device_sm_count(); }

Layout layout(int batch, int tokens, int max_new, int max_len, int heads, int kv_heads, int D,
              bool weights) {
  Layout l;
  const int G = heads / kv_heads;
  l.row_len = (max_len + 3) / 4 * 4;
  size_t at = 0;
  l.counters = at;
  at += round256(static_cast<size_t>(batch) * kv_heads * ((static_cast<size_t>(max_new) * G + 7) / 8) * 4);
  l.parts = at;
  at += round256(static_cast<size_t>(2) * grid_limit() * kMaxTiles * 8 * (D + 2) * 4);
  l.lse2 = at;
  if (weights) at += round256(static_cast<size_t>(tokens) * heads * 4);
  l.logits = at;
  if (weights)
    at += round256(static_cast<size_t>(batch) * heads * max_new * l.row_len * 4);
  l.total = at;
  return l;
}

template <int D, int NG, int NT>
cudaError_t run(const Kv4AttentionArgs& a, cudaStream_t stream) {
  constexpr int kStages = 2;
  using S = Shape<D, NG, NT, kStages>;
  const Layout l = layout(a.c.batch, a.tokens, a.max_new, a.max_len, a.heads, a.c.kv_heads, D,
                          a.weights_out != nullptr);
  Workspace ws;
  ws.counters = reinterpret_cast<uint32_t*>(a.workspace + l.counters);
  ws.lse2 = reinterpret_cast<float*>(a.workspace + l.lse2);
  ws.logits = reinterpret_cast<float*>(a.workspace + l.logits);
  ws.parts = reinterpret_cast<float*>(a.workspace + l.parts);
  ws.row_len = l.row_len;
  auto kern = a.weights_out != nullptr ? kv4_attention_kernel<D, NG, NT, kStages, true>
                                       : kv4_attention_kernel<D, NG, NT, kStages, false>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), S::total);
  if (e != cudaSuccess) return e;
  const int G = a.heads / a.c.kv_heads;
  const int64_t tiles = (static_cast<int64_t>(a.max_new) * G + S::kRows - 1) / S::kRows;
  const int64_t units = static_cast<int64_t>(a.c.batch) * a.c.kv_heads * tiles *
                        ((a.max_len + kUnit - 1) / kUnit + 1);
  const int64_t want = (units + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(want < grid_limit() ? want : grid_limit());
  e = launch_with_pdl(kern, dim3(grid), dim3(kWarps * 32), S::total, stream, a, ws);
  if (e != cudaSuccess || a.weights_out == nullptr) return e;
  return launch_with_pdl(kv4_weights_kernel,
                         dim3((a.max_len + 255) / 256, a.c.kv_heads, a.c.batch), dim3(256), 0,
                         stream, a, ws);
}

template <int D, int NG>
cudaError_t by_rows(const Kv4AttentionArgs& a, cudaStream_t stream) {
  const int rows = a.max_new * (a.heads / a.c.kv_heads);
  return rows <= 8 ? run<D, NG, 1>(a, stream) : run<D, NG, 2>(a, stream);
}

// Rows of a key/value head from which the prompts' path takes over.
constexpr int64_t kPromptRows = 33;

bool is_prompt(int max_new, int heads, int kv_heads) {
  return static_cast<int64_t>(max_new) * (heads / kv_heads) >= kPromptRows;
}

}  // namespace

size_t kv4_attention_workspace(int batch, int tokens, int max_new, int max_len, int heads,
                               int kv_heads, int head_dim, int group, bool weights) {
  if (is_prompt(max_new, heads, kv_heads))
    return kv4_prompt_workspace(batch, tokens, max_new, max_len, heads, kv_heads, head_dim, weights);
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
