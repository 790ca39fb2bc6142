// Attention of prompts over the 4-bit key/value cache: the tensor-memory path, for more rows
// (new token, query head) a key/value head than the few that kv4_attention.cu takes.
//
//   S = Q K_hat^T,  P = exp2(scale log2(e) S - m),  O = P V_hat,  out = O / rowsum(P)
//
// 4 D operations a visible (row, token) pair and one exponential: the tensor pipe bounds it. A unit
// of 256 rows and 128 tokens (D 128) needs 2176 cycles of multiplication; with both operands of
// the first product in shared memory it takes 2758, as reading them saturates it, and the whole
// loop took 2890 while P came under the tiles' powers of two alone (the kernel is 3 % slower with
// the rows' products). A prompt of 4096 tokens, 32 heads on 8: images 20.5 us, attention 120 us
// (0.60 of cuBLAS's BF16 rate on the visible pairs); 512 tokens behind 15872: 27 and 117 us.
//
// 1. kv4_prompt_images_kernel writes the sequence's keys and values, and the queries, as FP16
//    tiles in the swizzled order that tcgen05.mma reads: every later load is one contiguous bulk
//    copy, and a code is widened once instead of once a row tile (a 4096-token prompt has 64 of
//    them a head). Values come transposed, so that both products read K-major operands, rounded
//    to FP16 under a power of two a tile (scale, minimum and sum to 2^-11 of themselves; the
//    output's own rounding is 2^-8).
//    A tile whose tokens differ by 2^8 or more (a token that is larger than the rest would take
//    bits from them even in rows that do not see it) has powers of two a token, and the softmax a
//    slower body for it; 256 rows of queries that differ by 2^12 have them a row.
//    A key is exact: with c the code less 8, c s has at most 3 + 8 significant bits and is an
//    FP16 number; what is left, (min + 8 s) times the sum of q over the group, goes through 16
//    more columns, four a group, as FP16 pairs of high and low parts. Rounded keys put 3e-5 into
//    the accumulated weights, which are fp32.
// 2. kv4_prompt_kernel, one CTA an SM: 256 rows as two row halves of 128, each with a warpgroup
//    that owns one row a thread (no shuffles), over tiles of 128 tokens in a ring of four bulk
//    copies. One thread issues S = Q K^T (tensor memory, fp32) and O += P V with P read back from
//    tensor memory, the halves in turn, so that one half's softmax runs under the other's
//    products. P comes under the largest product of a probability and a tile's values that its row
//    has met, with 10 bits to spare; the running maximum may lag by 2^8 and that product by 2^5
//    before O is rescaled: P stays in FP16's range and the rescale is rare. The (sequence, head,
//    256-row tile) items, each as many units as it has visible token tiles, are cut into equal
//    ranges of units, one a CTA; an item that a boundary cuts is joined from fp32 parts by whoever
//    arrives last, in order.
// 3. With weights, kv4_prompt_weights_kernel makes S^T = K_hat Q^T from the same tiles, a thread
//    a token, and sums exp2(S - lse) along the row.
#include "kv4_common.cuh"
#include "kv4_prompt.h"

namespace w4k {
namespace {

constexpr int kTileKeys = 128;
constexpr int kTileRows = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct KeyMeta {
  float kf;  // a key's image times this is the key
  int ev;    // a value's image times 2^ev is the value; kByToken: as ws.tokens says
};
struct TokenMeta {
  float kf, ev;  // kf 0: the token's page is out of range, no row sees it
};
constexpr int kByToken = 1 << 20;
constexpr int kSpread = 8;  // exponents between a tile's tokens that one power of two bridges
// An fma takes the maximum off a logit (base 2) up to this size; beyond it the maximum's own
// rounding would be seen (and overflow P from 2^28 on), so the logit is rounded first, as the
// maximum was.
constexpr float kHuge = 1048576.f;
constexpr float kByRow = -1.f;
constexpr int kRowSpread = 12;  // the same between a tile's rows
// ev of a tile whose values are all 0: below any other's, so that it makes no row's product larger.
constexpr int kNoValue = -200;
// P reaches 2^kLift where its row's largest product is made, and 2^15 once that product lags.
constexpr int kLift = 10;

// Where a CTA begins: an item, the units of it before the CTA's range, and the range's size.
struct Start {
  int b, h, tile, before;
  uint32_t item_base, left;
  int units;  // of the item
  Kv4Seq s;
};
struct Plan {
  uint32_t total, ctas;  // units, and the CTAs that share them
  // items of `order` if whole items are dealt out, 0 if the units are cut into equal ranges
  uint32_t dealt;
};
// Up to this many (sequence, row tile) pairs may be put in order of their size.
constexpr int kOrdered = 512;

struct PromptWs {
  Plan* plan;         // [2]: of the row tiles, of the weights' key tiles
  Start* starts;      // [2][grid]
  Start* order;       // [kOrdered]: row tiles, longest first (b, tile, units and s)
  uint32_t* base;     // [batch + 1]: units before a sequence
  int32_t* pre;       // [batch, row_tiles + 1]: units of a head before a row tile
  KeyMeta* meta;      // [batch, kv_heads, key_tiles]
  TokenMeta* tokens;  // [batch, kv_heads, key_tiles, 128], of the tiles with kByToken
  // [batch, kv_heads, row_tiles, 256]: logit (base 2) per image product, without kf
  float* row_qf;
  // [batch, kv_heads, row_tiles]: the same of all rows, for the weights; kByRow: the weights go by
  // row_qf, as the rows have powers of two of their own or kHuge logits
  float* qf;
  uint8_t* q_img;     // [batch, kv_heads, row_tiles] x 256 (D + 16) FP16
  uint8_t* kv_img;    // [batch, kv_heads, key_tiles] x (K 128 (D + 16), V^T D 128) FP16
  uint32_t* counters; // [batch, kv_heads, row_tiles, 2], zeroed beside the images
  float* parts;       // [2 grid][2 halves] x (D + 2) 128
  // [batch, kv_heads, row_tiles, 256]: less the log-sum, base 2; -inf for a row that sees nothing
  float* lse2;
  // with weights, the same for the units of the token tiles (row tiles that see them)
  uint32_t* kbase;    // [batch + 1]
  int32_t* kpre;      // [batch, key_tiles + 1]
  uint32_t* kcounters;  // [batch, kv_heads, key_tiles], zeroed beside the images
  float* sums;        // [2 grid] x 128
  int key_tiles, row_tiles, grid;
};

template <int D>
struct Img {
  static constexpr uint32_t kMore = 16 * 2;                      // bytes of the 16 more columns
  static constexpr uint32_t kKCodes = kTileKeys * D * 2;         // one K tile without them
  static constexpr uint32_t kTile = kKCodes + kTileKeys * kMore; // with them
  static constexpr uint32_t kVTile = kTileKeys * D * 2;          // one V^T tile
  static constexpr uint32_t kPair = kTile + kVTile;
  static constexpr uint32_t kQCodes = kTileRows * D * 2;
  static constexpr uint32_t kQ = kQCodes + kTileRows * kMore;
};

// Units of a row tile: its key tiles, after kItemCost units that stand for the time an item costs
// beyond them (loading its queries, filling the pipeline, writing its rows). Without them the
// CTAs that get the short items at the beginning of a causal prompt finish last: a 4096-token
// prompt (32 heads) took 215 us, half of the CTAs having been done at 153.
constexpr int kItemCost = 2;
__device__ __forceinline__ int units_of(const Kv4Seq& s, int G, int rt) {
  const int last = min((rt + 1) * kTileRows, s.m * G) - 1;
  const int key = s.n - s.m + last / G;
  return kItemCost + (key < 0 ? 1 : key / kTileKeys + 1);
}

// ---- images ------------------------------------------------------------------------------
constexpr int kImgThreads = 512;

// Largest a and b (16 bits) of the block, a in the low half.
__device__ __forceinline__ uint32_t block_max(uint32_t a, uint32_t b, uint32_t* sm) {
  uint32_t v = __reduce_max_sync(0xffffffffu, a) | (__reduce_max_sync(0xffffffffu, b) << 16);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
#pragma unroll
  for (int i = 1; i < kImgThreads / 32; ++i) v = __vmaxu2(v, sm[i]);
  return v;
}
// Largest magnitude of eight BF16 values, as bits.
__device__ __forceinline__ uint32_t top_bits(const uint4& x) {
  const uint32_t t = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                              __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(t & 0xFFFFu, t >> 16);
}

// Exponent that brings a largest magnitude (fp32 bits, finite) to [2^14, 2^15).
__device__ __forceinline__ int up_of(uint32_t bits) {
  const int ex = static_cast<int>(bits >> 23);
  return ex == 0 ? 0 : min(max(141 - ex, -126), 126);
}

// Largest finite magnitude of a group's values, fp32 bits.
__device__ __forceinline__ uint32_t reach_bits(uint32_t param) {
  const float s = bf16_lo(param), m = bf16_hi(param);
  const uint32_t a = __float_as_uint(fabsf(m)), b = __float_as_uint(fabsf(fmaf(15.f, s, m)));
  return max(a >= 0x7F800000u ? 0u : a, b >= 0x7F800000u ? 0u : b);
}

__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// FP16 pairs (q - 8, q' - 8) of nibbles i and i + 4, exact.
__device__ __forceinline__ void centred_pairs(uint32_t w, uint32_t (&p)[4]) {
  code_pairs_f16(w, p);  // 1024 + q (even i) and 1024 + 16 q (odd i)
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = i % 2 == 0 ? fma_f16x2(p[i], 0x3C003C00u, 0xE408E408u)   // x - 1032
                      : fma_f16x2(p[i], 0x2C002C00u, 0xD480D480u);  // x / 16 - 72
}

// Three of the four more columns of a group: high and low FP16 parts of x.
__device__ __forceinline__ uint32_t high_low(float x) {
  const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
  return static_cast<uint32_t>(__half_as_ushort(hi)) |
         (static_cast<uint32_t>(__half_as_ushort(lo)) << 16);
}

// 128 tokens of one head: their records come into shared memory by bulk copies at once (a load
// for each word, with the images' stores between them, made every word wait for memory).
template <int D, int NG>
__device__ void key_tile(const Kv4AttentionArgs& a, const PromptWs& ws, int b, int h, int tile,
                         uint8_t* raw) {
  using R = Kv4Record<D, NG>;
  __shared__ uint32_t reach[2][kTileKeys];  // largest magnitudes of the tokens' keys and values
  __shared__ uint64_t bar;
  __shared__ uint32_t present;  // bit j: record j is there
  __shared__ uint32_t abort_flag;
  const int tid = threadIdx.x;
  const Kv4Seq seq = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
  const int key0 = tile * kTileKeys;
  const size_t at = (static_cast<size_t>(b) * a.c.kv_heads + h) * ws.key_tiles + tile;
  if (tid == 0 && ws.kbase != nullptr) ws.kcounters[at] = 0u;
  if (seq.m == 0 || key0 >= seq.n) return;
  if (tid == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  if (tid < 32) {
    const uint8_t* src = nullptr;
    if (tid < 8 && key0 + 16 * tid < seq.n)
      src = kv4_record(a.c, a.c.table, a.c.width, b, h, key0 / 16 + tid, R::kBytes);
    const uint32_t have = __ballot_sync(0xffffffffu, src != nullptr);
    if (tid == 0) {
      present = have;
      mbar_arrive_expect_tx(&bar, __popc(have) * R::kBytes);
    }
    __syncwarp();
    if (src != nullptr) bulk_load(raw + tid * R::kBytes, src, R::kBytes, &bar);
  }
  __syncthreads();
  if (!mbar_wait_bounded(&bar, 0u, &abort_flag, a.c.status, a.wait_limit_ns)) {
    volatile uint32_t no_abort = 0u;  // the copies land before the block exits
    mbar_wait_bounded(&bar, 0u, &no_abort, a.c.status, a.wait_limit_ns);
  }
  // what is not there, and tokens past the length, become 0
  for (int x = tid; x < 8 * 16 * NG; x += kImgThreads) {
    const int j = x / (16 * NG), w = x % (16 * NG);
    if (!((present >> j) & 1u) || key0 + 16 * j + w % 16 >= seq.n) {
      reinterpret_cast<uint32_t*>(raw + j * R::kBytes + R::kKParams)[w] = 0u;
      reinterpret_cast<uint32_t*>(raw + j * R::kBytes + R::kVParams)[w] = 0u;
    }
  }
  __syncthreads();
  if (tid < 2 * kTileKeys) {
    const uint32_t* params = reinterpret_cast<const uint32_t*>(
        raw + (tid % kTileKeys) / 16 * R::kBytes + (tid < kTileKeys ? R::kKParams : R::kVParams));
    uint32_t top = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) top = max(top, reach_bits(params[16 * g + tid % 16]));
    reach[tid / kTileKeys][tid % kTileKeys] = top;
  }
  __syncthreads();
  // exponents of the tile's largest token and of its smallest one that is not 0
  uint32_t tops[2];
  const int records = min(8, (seq.n - key0 + 15) / 16);
  bool by_token = present != (1u << records) - 1u;  // a page is out of range
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    uint32_t top = 0, low = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < kTileKeys; i += 32) {
      const uint32_t x = reach[y][i + tid % 32];
      top = max(top, x);
      low = min(low, x - 1u);  // 0 is the largest
    }
    tops[y] = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_min_sync(0xffffffffu, low);
    by_token = by_token || (tops[y] != 0u && (tops[y] >> 23) - (low >> 23) >= kSpread);
  }
  // keys reach [2^7, 2^8): 128 times a minimum + 8 s still is an FP16 number
  auto key_up = [](uint32_t top) { return max(up_of(top) - 7, -126); };
  const int kup = key_up(tops[0]), vup = up_of(tops[1]);
  if (tid == 0)
    ws.meta[at] = KeyMeta{pow2f(-kup), by_token ? kByToken : tops[1] == 0u ? kNoValue : -vup};
  if (by_token && tid < kTileKeys) {
    const uint32_t top = reach[1][tid];
    ws.tokens[at * kTileKeys + tid] =
        TokenMeta{(present >> (tid / 16)) & 1u ? pow2f(-key_up(reach[0][tid])) : 0.f,
                  static_cast<float>(top == 0u ? kNoValue : -up_of(top))};
  }
  const float kf_tile = pow2f(kup), vf_tile = pow2f(vup);
  auto key_factor = [&](int t) { return by_token ? pow2f(key_up(reach[0][t])) : kf_tile; };
  auto value_factor = [&](int t) { return by_token ? pow2f(up_of(reach[1][t])) : vf_tile; };
  uint8_t* kimg = ws.kv_img + at * Img<D>::kPair;
  uint8_t* vimg = kimg + Img<D>::kTile;
  constexpr int kWords = D / 8;
  for (int x = tid; x < kTileKeys * kWords; x += kImgThreads) {
    const int t = x / kWords, w = x % kWords, c = w / R::kBlocks, s = w % R::kBlocks;
    const int d = 32 * s + 8 * c;
    const uint8_t* rec = raw + (t / 16) * R::kBytes;
    const uint32_t word = reinterpret_cast<const uint32_t*>(rec)[(t % 16) * kWords + w];
    const uint32_t p =
        reinterpret_cast<const uint32_t*>(rec + R::kKParams)[16 * (d / R::kGroup) + t % 16];
    const float scale = bf16_lo(p) * key_factor(t);
    const uint32_t sc = f16x2_bits(scale, scale);
    uint32_t out[4];
    centred_pairs(word, out);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = mul_f16x2(out[i], sc);
    *reinterpret_cast<uint4*>(kimg + (d / 64) * (kTileKeys * 128) + t * 128 +
                              (((d % 64) / 8) ^ (t & 7)) * 16) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
  if (tid < kTileKeys) {
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float kf = key_factor(tid);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t p = reinterpret_cast<const uint32_t*>(
          raw + (tid / 16) * R::kBytes + R::kKParams)[16 * g + tid % 16];
      const uint32_t hl = high_low(fmaf(8.f, bf16_lo(p), bf16_hi(p)) * kf * 128.f);
      w[2 * g] = (hl & 0xFFFFu) * 0x10001u;  // high, high, low, 0
      w[2 * g + 1] = hl >> 16;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(kimg + Img<D>::kKCodes + i * (kTileKeys * 16) + tid * 16) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  // eight of a record's tokens, dims 32 blk + 4 r + 0..3
  for (int x = tid; x < 8 * 8 * R::kBlocks * 2; x += kImgThreads) {
    const int w = x % (8 * R::kBlocks), half = x / (8 * R::kBlocks) % 2, j = x / (16 * R::kBlocks);
    const int d0 = 32 * (w % R::kBlocks) + 4 * (w / R::kBlocks), g = d0 / R::kGroup;
    const uint8_t* rec = raw + j * R::kBytes;
    const uint2* params = reinterpret_cast<const uint2*>(rec + R::kVParams) + 8 * g + 4 * half;
    uint32_t out[4][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint2 two = params[p];
      uint32_t code[4];
      centred_pairs(reinterpret_cast<const uint32_t*>(rec + R::kV)[(4 * half + p) * 8 * R::kBlocks + w],
                    code);
      // P of a row that does not see a token is 0; 0 times a value that is not finite is not
      auto param = [&](float v) { return fabsf(v) <= 65504.f ? v : 0.f; };
      const int t = 16 * j + 8 * half + 2 * p;
      const float f0 = value_factor(t), f1 = value_factor(t + 1);
      const float s0 = bf16_lo(two.x) * f0, s1 = bf16_lo(two.y) * f1;
      const uint32_t sc = f16x2_bits(param(s0), param(s1));
      const uint32_t mn = f16x2_bits(param(fmaf(8.f, s0, bf16_hi(two.x) * f0)),
                                     param(fmaf(8.f, s1, bf16_hi(two.y) * f1)));
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i][p] = fma_f16x2(code[i], sc, mn);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = d0 + i;
      *reinterpret_cast<uint4*>(vimg + (j / 4) * (D * 128) + d * 128 +
                                (((j % 4) * 2 + half) ^ (d & 7)) * 16) =
          make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]);
    }
  }
}

// 256 rows of one head; the sign of the scale goes into them.
template <int D, int NG>
__device__ void row_tile(const Kv4AttentionArgs& a, const PromptWs& ws, int b, int h, int rt) {
  __shared__ uint32_t red[kImgThreads / 32];
  const Kv4Seq seq = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
  const int G = a.heads / a.c.kv_heads, rows = seq.m * G, row0 = rt * kTileRows;
  const size_t at = (static_cast<size_t>(b) * a.c.kv_heads + h) * ws.row_tiles + rt;
  if (threadIdx.x < 2) ws.counters[2 * at + threadIdx.x] = 0u;
  if (row0 >= rows) return;
  constexpr int kChunks = D / 8, kPer = kTileRows * kChunks / kImgThreads;
  constexpr int kStep = kImgThreads / kChunks;  // rows between a thread's chunks
  const int ch = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  // (token, head) of the thread's rows, one division for all of them
  int token = (row0 + r0) / G, head = (row0 + r0) % G;
  const int token_step = kStep / G, head_step = kStep % G;
  uint4 v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (row0 + r0 + i * kStep < rows)
      v[i] = __ldg(reinterpret_cast<const uint4*>(
          a.q + static_cast<int64_t>(seq.s0 + token) * a.q_stride + (h * G + head) * D + 8 * ch));
    token += token_step;
    head += head_step;
    if (head >= G) {
      head -= G;
      ++token;
    }
  }
  // the rows' largest magnitudes, BF16 bits, two rows a word; 0 for a row of infinities or NaN
  uint32_t tops[kPer / 2];
  uint32_t top = 0, less = 0;  // of all rows (in both halves); 0xFFFF less the smallest but 0
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    uint32_t t = top_bits(v[i]) | (top_bits(v[i + 1]) << 16);
#pragma unroll
    for (int o = 1; o < kChunks; o <<= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
    if ((t & 0xFFFFu) >= 0x7F80u) t &= 0xFFFF0000u;
    if (t >= 0x7F800000u) t &= 0xFFFFu;
    tops[i / 2] = t;
    top = __vmaxu2(top, t);
    if ((t & 0xFFFFu) != 0u) less = max(less, 0xFFFFu - (t & 0xFFFFu));
    if ((t >> 16) != 0u) less = max(less, 0xFFFFu - (t >> 16));
  }
  top = block_max(max(top & 0xFFFFu, top >> 16), less, red);
  less = top >> 16;
  top &= 0xFFFFu;
  const bool by_row = top != 0u && (top >> 7) - ((0xFFFFu - less) >> 7) >= kRowSpread;
  const int up_tile = up_of(top << 16);
  const float qf1 = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * kLog2e;
  const float sign = a.scale < 0.f ? -1.f : a.scale > 0.f ? 1.f : 0.f;
  const float f_tile = sign * pow2f(up_tile), qf_tile = qf1 * pow2f(-up_tile);
  if (threadIdx.x == 0) ws.qf[at] = by_row ? kByRow : qf_tile;
  uint8_t* img = ws.q_img + at * Img<D>::kQ;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r0 + i * kStep;
    float f = f_tile, qf = qf_tile;
    if (by_row) {
      const int up = up_of((tops[i / 2] >> (16 * (i % 2))) << 16);
      f = sign * pow2f(up);
      qf = qf1 * pow2f(-up);
    }
    if (ch == 0) ws.row_qf[at * kTileRows + r] = qf;
    const float q[8] = {bf16_lo(v[i].x) * f, bf16_hi(v[i].x) * f, bf16_lo(v[i].y) * f,
                        bf16_hi(v[i].y) * f, bf16_lo(v[i].z) * f, bf16_hi(v[i].z) * f,
                        bf16_lo(v[i].w) * f, bf16_hi(v[i].w) * f};
    *reinterpret_cast<uint4*>(img + (ch / 8) * (kTileRows * 128) + r * 128 +
                              ((ch % 8) ^ (r & 7)) * 16) =
        make_uint4(f16x2_bits(q[0], q[1]), f16x2_bits(q[2], q[3]), f16x2_bits(q[4], q[5]),
                   f16x2_bits(q[6], q[7]));
    // the group's sum of q over 128, which the keys' columns make up for
    constexpr int kLanes = kChunks / NG;
    float sum = ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (ch % kLanes == 0) {
      const int g = ch / kLanes;
      const uint32_t hl = high_low(sum * 0.0078125f);
      uint8_t* more = img + Img<D>::kQCodes + r * 16;
      // high, low, high, 0
      *reinterpret_cast<uint2*>(more + (g / 2) * (kTileRows * 16) + (g % 2) * 8) =
          make_uint2(hl, hl & 0xFFFFu);
      if (g == 0)
        for (int x2 = NG; x2 < 4; ++x2)
          *reinterpret_cast<uint2*>(more + (x2 / 2) * (kTileRows * 16) + (x2 % 2) * 8) =
              make_uint2(0u, 0u);
    }
  }
}

// Row tiles that see a token of key tile kt.
__device__ __forceinline__ int first_row_tile(const Kv4Seq& s, int G, int kt) {
  const int64_t row = static_cast<int64_t>(kt * kTileKeys - (s.n - s.m)) * G;
  return row <= 0 ? 0 : static_cast<int>(row / kTileRows);
}
// Units of a token tile in the weights' kernel.
__device__ __forceinline__ int key_units_of(const Kv4Seq& s, int G, int kt) {
  return max(1, (s.m * G + kTileRows - 1) / kTileRows - first_row_tile(s, G, kt));
}

// Largest i < n with x[i] <= u, x non-decreasing from 0.
template <typename T>
__device__ __forceinline__ int last_at_most(const T* x, int n, T u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (x[mid] <= u)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ uint32_t scan_add(uint32_t u) {  // inclusive, over the warp
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, u, o);
    if (lane >= o) u += x;
  }
  return u;
}

// Tables of units_of_tile(sequence, tile), a warp a sequence, and where each CTA of an equal cut
// begins: the kernels would need five loads one after the other to find it. The searches go through
// a copy of the tables in shared memory (`room` words at sm) where they fit.
template <typename F>
__device__ void plan(const Kv4AttentionArgs& a, Plan* out, Start* starts, int grid, uint32_t* base,
                     int32_t* pre_all, int width, int32_t* sm, int room, F units_of_tile) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool fits = static_cast<int64_t>(a.c.batch) * (width + 2) + 1 <= room;
  int32_t* sm_pre = sm;
  uint32_t* sm_base = reinterpret_cast<uint32_t*>(sm + a.c.batch * (width + 1));
  for (int b = warp; b < a.c.batch; b += kImgThreads / 32) {
    const Kv4Seq s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, b);
    const size_t row = static_cast<size_t>(b) * (width + 1);
    uint32_t at = 0;
    for (int t0 = 0; t0 <= width; t0 += 32) {
      const uint32_t u = t0 + lane < width ? units_of_tile(s, t0 + lane) : 0;
      const uint32_t upto = scan_add(u);
      if (t0 + lane <= width) {
        pre_all[row + t0 + lane] = at + upto - u;
        if (fits) sm_pre[row + t0 + lane] = at + upto - u;
      }
      at += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) {
      base[b] = at * a.c.kv_heads;
      if (fits) sm_base[b] = at * a.c.kv_heads;
    }
  }
  __syncthreads();
  const int32_t* pre_tab = fits ? sm_pre : pre_all;
  uint32_t* base_tab = fits ? sm_base : base;
  if (warp == 0) {
    uint32_t at = 0;
    for (int b0 = 0; b0 < a.c.batch; b0 += 32) {
      const uint32_t u = b0 + lane < a.c.batch ? base_tab[b0 + lane] : 0;
      const uint32_t upto = scan_add(u);
      if (b0 + lane < a.c.batch) base_tab[b0 + lane] = at + upto - u;
      at += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) base_tab[a.c.batch] = at;
  }
  __syncthreads();
  const uint32_t total = base_tab[a.c.batch], ctas = min(static_cast<uint32_t>(grid), total);
  if (threadIdx.x == 0) *out = Plan{total, ctas, 0};
  if (total == 0) return;
  const Shares shares(total, ctas);
  for (uint32_t i = threadIdx.x; i < ctas; i += kImgThreads) {
    const uint32_t u0 = shares.begin(i);
    Start x;
    x.b = last_at_most(base_tab, a.c.batch, u0);
    x.s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, x.b);
    const int32_t* pre = pre_tab + static_cast<size_t>(x.b) * (width + 1);
    const uint32_t off = u0 - base_tab[x.b], per_head = pre[width];
    x.h = static_cast<int>(off / per_head);
    const int in_head = static_cast<int>(off % per_head);
    x.tile = last_at_most(pre, width, in_head);
    x.before = in_head - pre[x.tile];
    x.units = pre[x.tile + 1] - pre[x.tile];
    x.item_base = u0 - x.before;
    x.left = shares.begin(i + 1) - u0;
    starts[i] = x;
  }
}

// Whole items, longest first, dealt out to and fro over the CTAs, where that comes out even: no
// item is then cut, and a cut costs its CTAs about 8 us in parts written and joined. For a
// 4096-token prompt (512 items of up to 34 units, 62 a CTA) the largest hand is 5 % above the
// mean.
__device__ void deal(const Kv4AttentionArgs& a, const PromptWs& ws) {
  __shared__ uint32_t units[kOrdered];
  __shared__ uint32_t count, largest;
  const int n = a.c.batch * ws.row_tiles;
  if (n > kOrdered) return;
  if (threadIdx.x == 0) count = largest = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kImgThreads) {
    const int32_t* pre = ws.pre + static_cast<size_t>(i / ws.row_tiles) * (ws.row_tiles + 1) +
                         i % ws.row_tiles;
    units[i] = pre[1] - pre[0];
    if (units[i] > 0) atomicAdd(&count, 1u);
    atomicMax(&largest, units[i]);
  }
  __syncthreads();
  const Plan p = *ws.plan;
  if (count * a.c.kv_heads < 2 * p.ctas ||
      static_cast<uint64_t>(largest) * p.ctas * 5 > static_cast<uint64_t>(p.total) * 3)
    return;
  for (int i = threadIdx.x; i < n; i += kImgThreads) {
    if (units[i] == 0) continue;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += units[j] > units[i] || (units[j] == units[i] && j < i);
    Start x = {};
    x.b = i / ws.row_tiles;
    x.tile = i % ws.row_tiles;
    x.units = units[i];
    x.s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, x.b);
    ws.order[rank] = x;
  }
  if (threadIdx.x == 0) ws.plan->dealt = count * a.c.kv_heads;
}

template <int D, int NG>
__global__ void __launch_bounds__(kImgThreads, 2)
    kv4_prompt_images_kernel(const Kv4AttentionArgs a, const PromptWs ws) {
  __shared__ __align__(128) uint8_t raw[8 * Kv4Record<D, NG>::kBytes];
  pdl_launch_dependents();
  pdl_wait();
  int64_t x = blockIdx.x;
  if (x == 0) {
    const int G = a.heads / a.c.kv_heads;
    plan(a, ws.plan, ws.starts, ws.grid, ws.base, ws.pre, ws.row_tiles,
         reinterpret_cast<int32_t*>(raw), static_cast<int>(sizeof(raw) / 4),
         [&](const Kv4Seq& s, int t) { return t * kTileRows < s.m * G ? units_of(s, G, t) : 0; });
    __syncthreads();
    deal(a, ws);
    return;
  }
  if (x == 1) {
    if (ws.kbase == nullptr) return;
    const int G = a.heads / a.c.kv_heads;
    plan(a, ws.plan + 1, ws.starts + ws.grid, ws.grid, ws.kbase, ws.kpre, ws.key_tiles,
         reinterpret_cast<int32_t*>(raw), static_cast<int>(sizeof(raw) / 4),
         [&](const Kv4Seq& s, int t) { return t * kTileKeys < s.n ? key_units_of(s, G, t) : 0; });
    return;
  }
  x -= 2;
  const int64_t bh = static_cast<int64_t>(a.c.batch) * a.c.kv_heads;
  if (x < bh * ws.row_tiles) {
    const int i = static_cast<int>(x / ws.row_tiles);
    row_tile<D, NG>(a, ws, i / a.c.kv_heads, i % a.c.kv_heads, static_cast<int>(x % ws.row_tiles));
    return;
  }
  x -= bh * ws.row_tiles;
  const int i = static_cast<int>(x / ws.key_tiles);
  key_tile<D, NG>(a, ws, i / a.c.kv_heads, i % a.c.kv_heads, static_cast<int>(x % ws.key_tiles),
                  raw);
}

// ---- tcgen05 -----------------------------------------------------------------------------
// Operands as the low words of shared-memory descriptors (address and leading offset); the high
// words are the layout's. Descriptors of neighbouring columns differ by an addition to the low
// word, so a product costs its issuing thread few instructions: with the descriptors put
// together anew for each one the issue, not the tensor pipe, set the pace (100 cycles a product
// of 64).
constexpr uint32_t kDescSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);  // see smem_desc_kmajor_sw128
// 16 K-major columns without swizzle: 8-row pieces of 128 bytes one after the other, the second 8
// columns the leading offset behind the first.
constexpr uint32_t kDescPlain = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t leading) {
  return ((saddr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16);
}
// D[tmem] (+)= A[smem] B[smem], FP16 in, fp32 sums.
template <uint32_t HIGH>
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(HIGH)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem].
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescSw128)
      : "memory");
}
// True in one lane, always the same; the whole warp comes here, so that the values the elected
// lane issues products with stay uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
// Instruction descriptor, kind::f16: fp32 accumulator, FP16 A and B, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// (x, y) = (x, y) * a + b
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, s, t;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 t, {%3, %3};\n\t"
      "fma.rn.f32x2 v, v, s, t;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// (x, y) = (x, y) * a + (b, c)
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c) {
  asm("{\n\t.reg .b64 v, s, t;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 t, {%3, %4};\n\t"
      "fma.rn.f32x2 v, v, s, t;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c));
}

constexpr int kRing = 4;
constexpr int kLoadWarp = 8, kMmaWarp = 9;  // after two warpgroups of row threads
// Three warpgroups of 168 registers a thread at launch; the row threads hold a row of S, so the
// third gives up what they take: 2 x 208 + 88 = 3 x 168.
constexpr int kPromptThreads = 384;
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
}
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
}

template <int D>
struct Smem {
  static constexpr uint32_t q_off = 0;
  static constexpr uint32_t ring_off = Img<D>::kQ;
  static constexpr uint32_t bar_off = ring_off + kRing * Img<D>::kTile;
  // full[R], empty[R], q_full, q_empty, s_full[2], p_full[2], o_full[2], wg[2], drain
  static constexpr uint32_t nbars = 2 * kRing + 11;
  static constexpr uint32_t misc_off = bar_off + nbars * 8;
  static constexpr uint32_t total = misc_off + 32;
  static constexpr uint32_t alloc = total + 1024;
};

// Halves of a row tile that have rows.
__device__ __forceinline__ int halves_of(const Kv4Seq& s, int G, int rt) {
  return s.m * G - rt * kTileRows > 128 ? 2 : 1;
}

// A segment: the part of one (sequence, head, row tile) in this CTA's range of units.
struct Segment {
  int b, h, rt;
  int units;   // of the item
  int tiles;   // of them key tiles, the last ones
  int lo, hi;  // key tiles in this segment; none where the range holds only the item's cost
  uint32_t item_base, left;
  uint32_t dealt, turn;  // items dealt out; turns of the deal that this CTA has had
  Kv4Seq s;
};

__device__ __forceinline__ void enter(Segment& g, int units, int first) {
  g.units = units;
  g.tiles = units - kItemCost;
  const int end = static_cast<int>(min(static_cast<uint32_t>(units), first + g.left));
  g.left -= end - first;
  g.lo = max(0, first - kItemCost);
  g.hi = max(0, end - kItemCost);
}
__device__ __forceinline__ bool advance(Segment& g, const Kv4AttentionArgs& a, const PromptWs& ws,
                                        uint32_t ctas, int G) {
  if (g.dealt != 0) {
    const uint32_t i = g.turn * ctas + (g.turn % 2 == 0 ? blockIdx.x : ctas - 1 - blockIdx.x);
    if (i >= g.dealt) return false;
    ++g.turn;
    const Start x = ws.order[i / a.c.kv_heads];
    g.b = x.b;
    g.rt = x.tile;
    g.h = i % a.c.kv_heads;
    g.s = x.s;
    g.units = x.units;
    g.tiles = g.hi = g.units - kItemCost;
    g.lo = 0;
    return true;
  }
  do {
    if (g.left == 0) return false;
    g.item_base += g.units;
    if (++g.rt * kTileRows >= g.s.m * G) {
      g.rt = 0;
      if (++g.h >= a.c.kv_heads) {
        g.h = 0;
        do {
          if (++g.b >= a.c.batch) return false;
          g.s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, g.b);
        } while (g.s.m == 0);
      }
    }
    enter(g, units_of(g.s, G, g.rt), 0);
  } while (g.lo >= g.hi);
  return true;
}
// This CTA's first segment; false if it has none.
__device__ __forceinline__ bool begin(Segment& g, const Kv4AttentionArgs& a, const PromptWs& ws,
                                      const Plan& plan, const Start& x, int G) {
  g.dealt = plan.dealt;
  g.turn = 0;
  if (g.dealt != 0) return advance(g, a, ws, plan.ctas, G);
  g.b = x.b;
  g.h = x.h;
  g.rt = x.tile;
  g.s = x.s;
  g.item_base = x.item_base;
  g.left = x.left;
  enter(g, x.units, x.before);
  return g.lo < g.hi || advance(g, a, ws, plan.ctas, G);
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    kv4_prompt_kernel(const Kv4AttentionArgs a, const PromptWs ws) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar_off);
  uint64_t* empty = full + kRing;
  uint64_t* q_full = empty + kRing;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;  // a half's S is there, and its products before are done
  uint64_t* p_full = s_full + 2;   // a half's P is there, its S read, its O rescaled
  uint64_t* o_full = p_full + 2;   // a half's segment is complete
  uint64_t* wg_bar = o_full + 2;
  uint64_t* drain = wg_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  volatile uint32_t* arrived = tmem_holder + 2;  // [2]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.heads / a.c.kv_heads;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&wg_bar[i], 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();

  const Plan plan = ws.plan[0];
  const uint32_t me = blockIdx.x;
  const Start start = ws.starts[me];  // not written past plan.ctas, and not used there
  Segment g;
  const bool some = me < plan.ctas && begin(g, a, ws, plan, start, G);
  uint32_t* status = a.c.status;
  const uint64_t limit = a.wait_limit_ns;
  auto item = [&](const Segment& x) {
    return (static_cast<size_t>(x.b) * a.c.kv_heads + x.h) * ws.row_tiles + x.rt;
  };

  if (warp >= 8) {
    give_registers();
    if (some && warp == kLoadWarp) {
      if (lane == 0) {
        int n = 0, segs = 0;  // tiles loaded, segments begun
        bool ok = true;
        auto load = [&](const uint8_t* src, uint32_t bytes) {
          const int s = n % kRing;
          if (n >= kRing)
            ok = mbar_wait_bounded(&empty[s], (n / kRing - 1) & 1u, abort_flag, status, limit);
          if (!ok) return;
          mbar_arrive_expect_tx(&full[s], bytes);
          bulk_load(smem + L::ring_off + s * Img<D>::kTile, src, bytes, &full[s]);
          ++n;
        };
        do {
          if (segs > 0) ok = mbar_wait_bounded(q_empty, (segs - 1) & 1u, abort_flag, status, limit);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full, Img<D>::kQ);
          bulk_load(smem + L::q_off, ws.q_img + item(g) * Img<D>::kQ, Img<D>::kQ, q_full);
          ++segs;
          const uint8_t* kv = ws.kv_img + (static_cast<size_t>(g.b) * a.c.kv_heads + g.h) *
                                              ws.key_tiles * Img<D>::kPair;
          for (int i = g.lo; i < g.hi && ok; ++i) {
            const uint8_t* src = kv + static_cast<size_t>(i) * Img<D>::kPair;
            load(src, Img<D>::kTile);
            if (ok) load(src + Img<D>::kTile, Img<D>::kVTile);
          }
        } while (ok && advance(g, a, ws, plan.ctas, G));
        if (!ok) {  // copies in flight land before the CTA exits
          volatile uint32_t no_abort = 0u;
          for (int i = max(0, n - kRing); i < n; ++i)
            mbar_wait_bounded(&full[i % kRing], (i / kRing) & 1u, &no_abort, status, limit);
          if (segs > 0) mbar_wait_bounded(q_full, (segs - 1) & 1u, &no_abort, status, limit);
        }
      }
    } else if (some && warp == kMmaWarp) {
      constexpr uint32_t s_idesc = idesc_f16_f32(128, kTileKeys), o_idesc = idesc_f16_f32(128, D);
      const uint32_t q_s = desc_low(smem_addr(smem + L::q_off), 16);
      const uint32_t q_more = desc_low(smem_addr(smem + L::q_off) + Img<D>::kQCodes, kTileRows * 16);
      const uint32_t ring = desc_low(smem_addr(smem + L::ring_off), 16);
      const uint32_t ring_more =
          desc_low(smem_addr(smem + L::ring_off) + Img<D>::kKCodes, kTileKeys * 16);
      int n = 0, segs = 0, steps = 0, steps_1 = 0;  // tiles of all halves, of second halves
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait_bounded(bar, parity, abort_flag, status, limit);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      auto s_mma = [&](int half, int slot) {
        const uint32_t k_s = ring + slot * (Img<D>::kTile >> 4), q_h = q_s + half * (16384 >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss<kDescSw128>(tmem + half * 128,
                                q_h + (((kk / 4) * (kTileRows * 128) + (kk % 4) * 32) >> 4),
                                k_s + (((kk / 4) * (kTileKeys * 128) + (kk % 4) * 32) >> 4), s_idesc,
                                kk != 0);
        tc_mma_ss<kDescPlain>(tmem + half * 128, q_more + half * (2048 >> 4),
                              ring_more + slot * (Img<D>::kTile >> 4), s_idesc, 1u);
      };
      auto o_mma = [&](int half, int slot, bool first) {
        const uint32_t v_s = ring + slot * (Img<D>::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kTileKeys / 16; ++kk)
          tc_mma_ts(tmem + 256 + half * D, tmem + half * 128 + kk * 8,
                    v_s + (((kk / 4) * (D * 128) + (kk % 4) * 32) >> 4), o_idesc,
                    kk != 0 || !first);
      };
      do {
        if (!wait(q_full, segs & 1u)) break;
        ++segs;
        if (!wait(&full[n % kRing], (n / kRing) & 1u)) break;
        tc_fence_after_sync();
        const int halves = halves_of(g.s, G, g.rt);
        if (elect_one()) {
          s_mma(0, n % kRing);
          tc_commit(&s_full[0]);
          if (halves == 2) {
            s_mma(1, n % kRing);
            tc_commit(&s_full[1]);
          }
          tc_commit(&empty[n % kRing]);
          if (g.hi - g.lo == 1) tc_commit(q_empty);
        }
        __syncwarp();
        ++n;
        for (int i = g.lo; i < g.hi && ok; ++i) {
          const bool more = i + 1 < g.hi;
          const int v_slot = n % kRing, k_slot = (n + 1) % kRing;
          if (!wait(&full[v_slot], (n / kRing) & 1u)) break;
          if (more && !wait(&full[k_slot], ((n + 1) / kRing) & 1u)) break;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half >= halves) break;
            const bool last = half + 1 == halves;
            if (!wait(&p_full[half], (half == 0 ? steps : steps_1) & 1u)) break;
            tc_fence_after_sync();
            if (elect_one()) {
              o_mma(half, v_slot, i == g.lo);
              if (last) tc_commit(&empty[v_slot]);
              if (more) s_mma(half, k_slot);
              tc_commit(more ? &s_full[half] : &o_full[half]);
              if (more && last) {
                tc_commit(&empty[k_slot]);
                if (i + 2 == g.hi) tc_commit(q_empty);
              }
            }
            __syncwarp();
          }
          n += more ? 2 : 1;
          ++steps;
          if (halves == 2) ++steps_1;
        }
      } while (ok && advance(g, a, ws, plan.ctas, G));
      if (elect_one()) tc_commit(drain);
      volatile uint32_t no_abort = 0u;
      mbar_wait_bounded(drain, 0u, &no_abort, status, limit);
    }
  } else {
    take_registers();
    if (some) {
      const int half = warp >> 2, row = threadIdx.x & 127;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + half * 128, t_o = tmem + lanes + 256 + half * D;
      uint32_t s_phase = 0, o_phase = 0, wg_phase = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t& phase) {
        ok = ok && mbar_wait_bounded(bar, phase & 1u, abort_flag, status, limit);
        ok = __all_sync(0xffffffffu, ok);
        ++phase;
        tc_fence_after_sync();
        return ok;
      };
      auto wg_sync = [&]() {
        mbar_arrive(&wg_bar[half]);
        return wait(&wg_bar[half], wg_phase);
      };
      do {
        const Kv4Seq seq = g.s;
        if (half >= halves_of(seq, G, g.rt)) {
          if (ws.lse2 != nullptr) ws.lse2[item(g) * kTileRows + 128 + row] = -INFINITY;
          continue;
        }
        const int rows = seq.m * G, R = g.rt * kTileRows + half * 128 + row;
        const int last_key = R < rows ? seq.n - seq.m + R / G : -1;
        // first key that some row of this half does not see
        const int first_row = g.rt * kTileRows + half * 128;
        const int clear = first_row + 127 < rows ? seq.n - seq.m + first_row / G + 1 : 0;
        const float qf = ws.row_qf[item(g) * kTileRows + half * 128 + row];
        const size_t tile0 = (static_cast<size_t>(g.b) * a.c.kv_heads + g.h) * ws.key_tiles;
        const KeyMeta* meta = ws.meta + tile0;
        KeyMeta km = meta[g.lo];
        // the running maximum; the sum of probabilities under it; and, under it too, the exponent
        // (a whole number) that O and the row's products come under
        float m = -INFINITY, l = 0.f, e = 0.f;
        bool huge = false;  // a row of the warp has met a logit beyond kHuge
        // a tile whose largest logit (base 2) is t, and whose largest product is `product`
        auto raises = [&](float t, float product) {
          return t > m + 8.f || product - m > e + 15.f;
        };
        auto raise = [&](float t, float product, bool first) {
          float f = 1.f;
          if (raises(t, product)) {
            const float top = fmaxf(m, t), old = e + (m - top);
            l *= ex2(m - top);
            const float now_e = fmaxf(ceilf(old), ceilf(product - top) - kLift);
            f = ex2(old - now_e);
            m = top;
            e = now_e;
          }
          if (!first && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld_16cols(t_o + 16 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_16cols(t_o + 16 * c, o);
            }
          }
        };
        auto is_huge = [](float t) { return fabsf(t) > kHuge && t != -INFINITY; };
        auto hand_over = [&]() {
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[half]);
        };
        for (int i = g.lo; i < g.hi; ++i) {
          const KeyMeta now = km;
          if (i + 1 < g.hi) km = meta[i + 1];
          const float cf = fmaxf(qf * now.kf, 1e-37f);
          if (!wait(&s_full[half], s_phase)) break;
          const int see = last_key - i * kTileKeys;  // columns up to this one are visible
          if (now.ev != kByToken && !huge) {
            float s[128];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tmem_ld_32cols(t_s + 32 * c, reinterpret_cast<uint32_t*>(s) + 32 * c);
            tmem_ld_wait();
            if ((i + 1) * kTileKeys > clear) {
#pragma unroll
              for (int j = 0; j < 128; ++j) s[j] = j <= see ? s[j] : -INFINITY;
            }
            float top[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) top[x] = max3(s[x], s[x + 8], s[x + 16]);
#pragma unroll
            for (int j = 24; j < 120; j += 16) {
#pragma unroll
              for (int x = 0; x < 8; ++x) top[x] = max3(top[x], s[j + x], s[j + 8 + x]);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) top[x] = fmaxf(top[x], s[120 + x]);
            const float best = max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]),
                                    fmaxf(top[6], top[7]));
            const float ev = static_cast<float>(now.ev);
            const float t = best * cf;  // -inf stays -inf: cf is positive
            if (__any_sync(0xffffffffu, raises(t, t + ev) || is_huge(t))) {
              huge = __any_sync(0xffffffffu, is_huge(t));
              if (!huge) raise(t, t + ev, i == g.lo);
            }
            if (!huge) {
              // P is the probability (under m) times 2^-down, l takes that out again. Past 2^60 the
              // tile's values are nothing beside the row's products and P is 0; before 2^-126 its
              // probabilities are nothing beside l
              const float down = fminf(e - ev, 60.f);
              const float bias = -((m == -INFINITY ? 0.f : m) + down);
              const float undo = pow2f(static_cast<int>(fmaxf(down, -126.f)));
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t p[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  float x = s[64 * c + 2 * j], y = s[64 * c + 2 * j + 1];
                  fma2(x, y, cf, bias);
                  x = ex2(x);
                  y = ex2(y);
                  add2(acc[2 * (j & 1)], acc[2 * (j & 1) + 1], x, y);
                  p[j] = f16x2_bits(x, y);
                }
                tmem_st_32cols(t_s + 32 * c, p);
              }
              hand_over();
              l = fmaf((acc[0] + acc[1]) + (acc[2] + acc[3]), undo, l);
              continue;
            }
          }
          // powers of two a token, or logits rounded before the maximum comes off: S is read
          // twice, 32 columns at a time
          const TokenMeta* tok = ws.tokens + (tile0 + i) * kTileKeys;
          const TokenMeta tile{now.kf, static_cast<float>(now.ev)};
          auto token = [&](int j) { return now.ev == kByToken ? tok[j] : tile; };
          uint32_t x[32];
          auto logits = [&](int c) {
            tmem_ld_32cols(t_s + 32 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float kf = token(32 * c + j).kf;
              x[j] = __float_as_uint(
                  32 * c + j <= see && kf != 0.f
                      ? __fmul_rn(__uint_as_float(x[j]), fmaxf(qf * kf, 1e-37f)) : -INFINITY);
            }
          };
          float t = -INFINITY, product = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            logits(c);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              t = fmaxf(t, __uint_as_float(x[j]));
              product = fmaxf(product, __uint_as_float(x[j]) + token(32 * c + j).ev);
            }
          }
          huge = huge || __any_sync(0xffffffffu, is_huge(t));
          raise(t, product, i == g.lo);
          const float under = m == -INFINITY ? 0.f : m;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {  // P's columns are behind those of S still to be read
            logits(c);
            float acc = 0.f, p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float y = __uint_as_float(x[j]) - under;
              acc += ex2(y);
              p[j] = ex2(y + (token(32 * c + j).ev - e));
            }
            l += acc;
            uint32_t pairs[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) pairs[j] = f16x2_bits(p[2 * j], p[2 * j + 1]);
            tmem_st_16cols(t_s + 16 * c, pairs);
          }
          hand_over();
        }
        if (!ok || !wait(&o_full[half], o_phase)) break;
        if (huge && ws.lse2 != nullptr && lane == 0) ws.qf[item(g)] = kByRow;
        // ---- O is complete
        const float vf = scalbnf(1.f, static_cast<int>(e));
        const bool whole = g.lo == 0 && g.hi == g.tiles;
        const bool have = R < rows;
        const int64_t at =
            have ? static_cast<int64_t>(seq.s0 + R / G) * a.heads + g.h * G + R % G : 0;
        auto finish = [&](float mm, float ll) {
          const float lse2 = ll == 0.f ? -INFINITY : mm + log2f(ll);
          if (have && a.lse != nullptr) a.lse[at] = lse2 * kLn2;
          if (ws.lse2 != nullptr)
            ws.lse2[item(g) * kTileRows + half * 128 + row] =
                have && lse2 != -INFINITY ? -lse2 : -INFINITY;
        };
        auto store32 = [&](int c, const float* v, float inv) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = inv == 0.f ? 0u : bf16x2_bits(v[2 * j] * inv, v[2 * j + 1] * inv);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(a.out + at * D + 32 * c + 8 * j) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        };
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32cols(t_o + 32 * c, o);
            tmem_ld_wait();
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]) * vf;
            if (have) store32(c, v, inv);
          }
          finish(m, l);
        } else {
          constexpr size_t kPart = static_cast<size_t>(D + 2) * 128;
          float* base = ws.parts + ((2 * me + (g.lo == 0 ? 1 : 0)) * 2 + half) * kPart;
          float* part = base + 4 * row;
          float2* ml = reinterpret_cast<float2*>(base + D * 128);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32cols(t_o + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              __stcg(reinterpret_cast<float4*>(part) + (8 * c + j / 4) * 128,
                     make_float4(__uint_as_float(o[j]) * vf, __uint_as_float(o[j + 1]) * vf,
                                 __uint_as_float(o[j + 2]) * vf, __uint_as_float(o[j + 3]) * vf));
          }
          __stcg(ml + row, make_float2(m, l));
          const Shares shares(plan.total, plan.ctas);
          const uint32_t i0 = shares.of(g.item_base + kItemCost);
          const uint32_t i1 = shares.of(g.item_base + g.units - 1);
          if (!wg_sync()) break;
          if (row == 0) {
            __threadfence();  // the half's writes, which the barrier has ordered before this
            uint32_t* cnt = ws.counters + item(g) * 2 + half;
            const bool last = atomicAdd(cnt, 1u) == i1 - i0;
            if (last) *cnt = 0u;
            __threadfence();
            arrived[half] = last ? 1u : 0u;
          }
          if (!wg_sync()) break;
          if (arrived[half]) {
            // the parts in the CTAs' order; this one's is still in tensor memory
            auto part_of = [&](uint32_t i) {
              return ws.parts + ((2 * i + (i == i0 ? 1 : 0)) * 2 + half) * kPart;
            };
            auto ml_of = [&](uint32_t i) {
              return i == me ? make_float2(m, l)
                             : __ldcg(reinterpret_cast<const float2*>(part_of(i) + D * 128) + row);
            };
            float mm = -INFINITY, ll = 0.f;
            for (uint32_t i = i0; i <= i1; i += 4) {
              float2 x[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[j] = i + j <= i1 ? ml_of(i + j) : make_float2(-INFINITY, 0.f);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (x[j].x == -INFINITY) continue;
                const float top = fmaxf(mm, x[j].x);
                ll = fmaf(ll, ex2(mm - top), x[j].y * ex2(x[j].x - top));
                mm = top;
              }
            }
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              float v[64];
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] = 0.f;
              for (uint32_t i = i0; i <= i1; ++i) {
                const float x = ml_of(i).x, w = x == -INFINITY ? 0.f : ex2(x - mm);
                if (i == me) {
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    uint32_t o[16];
                    tmem_ld_16cols(t_o + 64 * c + 16 * z, o);
                    tmem_ld_wait();
                    if (w != 0.f) {
#pragma unroll
                      for (int j = 0; j < 16; ++j)
                        v[16 * z + j] = fmaf(__uint_as_float(o[j]) * vf, w, v[16 * z + j]);
                    }
                  }
                  continue;
                }
                const float4* src = reinterpret_cast<const float4*>(part_of(i)) + row;
                float4 t[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) t[j] = __ldcg(src + (16 * c + j) * 128);
                if (w != 0.f) {
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    v[4 * j] = fmaf(t[j].x, w, v[4 * j]);
                    v[4 * j + 1] = fmaf(t[j].y, w, v[4 * j + 1]);
                    v[4 * j + 2] = fmaf(t[j].z, w, v[4 * j + 2]);
                    v[4 * j + 3] = fmaf(t[j].w, w, v[4 * j + 3]);
                  }
                }
              }
              if (have) {
                store32(2 * c, v, inv);
                store32(2 * c + 1, v + 32, inv);
              }
            }
            finish(mm, ll);
          }
          if (!wg_sync()) break;  // `arrived` is read before it is written again
        }
      } while (advance(g, a, ws, plan.ctas, G));
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ---- weights -----------------------------------------------------------------------------
// Units are (row tile, token tile) pairs, token tile by token tile, cut evenly over the CTAs. 16
// warps: a thread a token (TMEM lane) and a quarter of a row tile's 256 columns; S^T is
// double-buffered in tensor memory, and a row tile's log-sums come as one more bulk copy. A token
// tile that a boundary cuts is joined from its parts (128 sums) by whoever arrives last, in order.
//
// A unit's products take 1490 cycles, with its 75 KB of loads 1750, a thread's way through 64
// exponentials and sums 2300 (1.2 us a unit: 78 us for a prompt of 4096 tokens of 32 heads on 8,
// 262 us for 8192). Eight warps of 128 columns each took 84 and 286 us, with a barrier a unit and
// the log-sums fetched by each thread 107 and 380; the next columns' load ahead of the sums spills
// at sixteen warps.
constexpr int kSumWarps = 16;
constexpr int kSumParts = kSumWarps / 4;
constexpr int kSumCols = kTileRows / kSumParts;
// The log-sums' ring. Unit n's are written once unit n - 2's products are made; those waited until
// every warp had read unit n - 4's, so unit n - 8's are done with.
constexpr int kLseRing = 8;
constexpr int kSumThreads = kSumWarps * 32;
constexpr int kWeightThreads = kSumThreads + 64;

template <int D>
struct WeightSmem {
  static constexpr uint32_t k_off = 0;
  static constexpr uint32_t q_off = 2 * Img<D>::kTile;
  static constexpr uint32_t lse_off = q_off + 2 * Img<D>::kQ;         // [kLseRing][256]
  static constexpr uint32_t sum_off = lse_off + kLseRing * kTileRows * 4;  // [parts - 1][128]
  static constexpr uint32_t bar_off = sum_off + (kSumParts - 1) * 128 * 4;
  // k_full[2], k_empty[2], q_full[2], q_empty[2], s_full[2], s_empty[2], lse_full[8], drain
  static constexpr uint32_t misc_off = bar_off + (13 + kLseRing) * 8;
  static constexpr uint32_t total = misc_off + 16;
  static constexpr uint32_t alloc = total + 1024;
};

__device__ __forceinline__ void sum_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSumThreads) : "memory");
}

struct KeySegment {
  int b, h, kt;
  int units;   // row tiles of the token tile
  int lo, hi;  // of them in this segment
  int first;   // first row tile
  uint32_t item_base, left;
  Kv4Seq s;
};
__device__ __forceinline__ void enter(KeySegment& g, int units, int G, int at) {
  g.units = units;
  g.first = first_row_tile(g.s, G, g.kt);
  g.lo = at;
  g.hi = static_cast<int>(min(static_cast<uint32_t>(units), at + g.left));
  g.left -= g.hi - g.lo;
}
__device__ __forceinline__ bool advance(KeySegment& g, const Kv4AttentionArgs& a, int G) {
  if (g.left == 0) return false;
  g.item_base += g.units;
  if (++g.kt * kTileKeys >= g.s.n) {
    g.kt = 0;
    if (++g.h >= a.c.kv_heads) {
      g.h = 0;
      do {
        if (++g.b >= a.c.batch) return false;
        g.s = kv4_sequence(a.c, a.starts, a.tokens, a.max_new, a.max_len, g.b);
      } while (g.s.n == 0);
    }
  }
  enter(g, key_units_of(g.s, G, g.kt), G, 0);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1)
    kv4_prompt_weights_kernel(const Kv4AttentionArgs a, const PromptWs ws) {
  using L = WeightSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::bar_off);
  uint64_t *k_empty = k_full + 2, *q_full = k_empty + 2, *q_empty = q_full + 2,
           *s_full = q_empty + 2, *s_empty = s_full + 2, *lse_full = s_empty + 2,
           *drain = lse_full + kLseRing;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  volatile uint32_t* arrived = tmem_holder + 2;
  float* lse_s = reinterpret_cast<float*>(smem + L::lse_off);
  float* sum_s = reinterpret_cast<float*>(smem + L::sum_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.heads / a.c.kv_heads;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSumWarps);
    }
    for (int i = 0; i < kLseRing; ++i) mbar_init(&lse_full[i], 1);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == kSumWarps + 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();

  const Plan plan = ws.plan[1];
  const uint32_t me = blockIdx.x;
  const bool some = me < plan.ctas;
  KeySegment g;
  if (some) {
    const Start x = ws.starts[ws.grid + me];
    g.b = x.b;
    g.h = x.h;
    g.kt = x.tile;
    g.s = x.s;
    g.item_base = x.item_base;
    g.left = x.left;
    enter(g, x.units, G, x.before);
  }
  uint32_t* status = a.c.status;
  const uint64_t limit = a.wait_limit_ns;
  auto head = [&]() { return static_cast<size_t>(g.b) * a.c.kv_heads + g.h; };
  if (!some) {
  } else if (warp == kSumWarps) {
    if (lane == 0) {
      bool ok = true;
      int n = 0, segs = 0;
      do {
        const int ks = segs & 1;
        if (segs >= 2)
          ok = mbar_wait_bounded(&k_empty[ks], (segs / 2 - 1) & 1u, abort_flag, status, limit);
        if (!ok) break;
        mbar_arrive_expect_tx(&k_full[ks], Img<D>::kTile);
        bulk_load(smem + L::k_off + ks * Img<D>::kTile,
                  ws.kv_img + (head() * ws.key_tiles + g.kt) * Img<D>::kPair, Img<D>::kTile,
                  &k_full[ks]);
        ++segs;
        for (int i = g.lo; i < g.hi; ++i, ++n) {
          const int s = n & 1;
          if (n >= 2)
            ok = mbar_wait_bounded(&q_empty[s], (n / 2 - 1) & 1u, abort_flag, status, limit);
          if (!ok) break;
          const size_t tile = head() * ws.row_tiles + g.first + i;
          const int z = n % kLseRing;
          mbar_arrive_expect_tx(&lse_full[z], kTileRows * 4);
          bulk_load(lse_s + z * kTileRows, ws.lse2 + tile * kTileRows, kTileRows * 4, &lse_full[z]);
          mbar_arrive_expect_tx(&q_full[s], Img<D>::kQ);
          bulk_load(smem + L::q_off + s * Img<D>::kQ,
                    ws.q_img + tile * Img<D>::kQ, Img<D>::kQ, &q_full[s]);
        }
      } while (ok && advance(g, a, G));
      if (!ok) {  // copies in flight land before the CTA exits
        volatile uint32_t no_abort = 0u;
        for (int i = max(0, segs - 2); i < segs; ++i)
          mbar_wait_bounded(&k_full[i & 1], (i / 2) & 1u, &no_abort, status, limit);
        for (int i = max(0, n - 2); i < n; ++i)
          mbar_wait_bounded(&q_full[i & 1], (i / 2) & 1u, &no_abort, status, limit);
        for (int i = max(0, n - kLseRing); i < n; ++i)
          mbar_wait_bounded(&lse_full[i % kLseRing], (i / kLseRing) & 1u, &no_abort, status, limit);
      }
    }
  } else if (warp == kSumWarps + 1) {
    constexpr uint32_t idesc = idesc_f16_f32(128, kTileRows);
    bool ok = true;
    int n = 0, segs = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && mbar_wait_bounded(bar, parity, abort_flag, status, limit);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    do {
      const int ks = segs & 1;
      if (!wait(&k_full[ks], (segs / 2) & 1u)) break;
      ++segs;
      const uint32_t k_at = smem_addr(smem + L::k_off) + ks * Img<D>::kTile;
      const uint32_t k_s = desc_low(k_at, 16);
      const uint32_t k_more = desc_low(k_at + Img<D>::kKCodes, kTileKeys * 16);
      for (int i = g.lo; i < g.hi; ++i, ++n) {
        const int s = n & 1;
        if (!wait(&q_full[s], (n / 2) & 1u)) break;
        if (n >= 2 && !wait(&s_empty[s], (n / 2 - 1) & 1u)) break;
        tc_fence_after_sync();
        const uint32_t q_at = smem_addr(smem + L::q_off) + s * Img<D>::kQ;
        const uint32_t q_s = desc_low(q_at, 16);
        const uint32_t q_more = desc_low(q_at + Img<D>::kQCodes, kTileRows * 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma_ss<kDescSw128>(tmem + s * 256,
                                  k_s + (((kk / 4) * (kTileKeys * 128) + (kk % 4) * 32) >> 4),
                                  q_s + (((kk / 4) * (kTileRows * 128) + (kk % 4) * 32) >> 4), idesc,
                                  kk != 0);
          tc_mma_ss<kDescPlain>(tmem + s * 256, k_more, q_more, idesc, 1u);
          tc_commit(&q_empty[s]);
          tc_commit(&s_full[s]);
          if (i + 1 == g.hi) tc_commit(&k_empty[ks]);
        }
        __syncwarp();
      }
    } while (ok && advance(g, a, G));
    if (elect_one()) tc_commit(drain);
    volatile uint32_t no_abort = 0u;
    mbar_wait_bounded(drain, 0u, &no_abort, status, limit);
  } else {
    const int part = warp >> 2;  // columns kSumCols part ..
    const uint32_t t_s =
        tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + part * kSumCols;
    bool ok = true;
    int n = 0;
    do {
      const int key = g.kt * kTileKeys + (warp & 3) * 32 + lane;
      const size_t tile = head() * ws.key_tiles + g.kt;
      const KeyMeta km = ws.meta[tile];
      const float kf = km.ev == kByToken
                           ? ws.tokens[tile * kTileKeys + key % kTileKeys].kf
                           : km.kf;
      float acc = 0.f;
      auto qf_of = [&](int i) { return ws.qf[head() * ws.row_tiles + g.first + i]; };
      // rows that do not see the lane's token, and the first tile whose rows see all of them
      const int64_t need = static_cast<int64_t>(key - (g.s.n - g.s.m)) * G;
      const int64_t last =
          static_cast<int64_t>(g.kt * kTileKeys + kTileKeys - 1 - (g.s.n - g.s.m)) * G;
      const int clear =
          static_cast<int>(max(static_cast<int64_t>(0), (last + kTileRows - 1) / kTileRows));
      float qf_next = g.lo < g.hi ? qf_of(g.lo) : 0.f;
      for (int i = g.lo; i < g.hi; ++i, ++n) {
        const int s = n & 1, rt = g.first + i;
        const float qf = qf_next;
        const float cf = fmaxf(qf * kf, 1e-37f);
        if (i + 1 < g.hi) qf_next = qf_of(i + 1);
        ok = ok && mbar_wait_bounded(&lse_full[n % kLseRing], (n / kLseRing) & 1u, abort_flag,
                                     status, limit) &&
             mbar_wait_bounded(&s_full[s], (n / 2) & 1u, abort_flag, status, limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc_fence_after_sync();
        const float* lse = lse_s + (n % kLseRing) * kTileRows + part * kSumCols;
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        if (qf == kByRow) {
          // a factor a row, and logits rounded before the log-sum comes off, as it was made
          const float* rows =
              ws.row_qf + (head() * ws.row_tiles + rt) * kTileRows + part * kSumCols;
          const int64_t hide = need - static_cast<int64_t>(rt) * kTileRows - part * kSumCols;
#pragma unroll 1
          for (int c = 0; c < kSumCols; c += 16) {
            float x[16];
            tmem_ld_16cols(t_s + s * 256 + c, reinterpret_cast<uint32_t*>(x));
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float f = fmaxf(rows[c + j] * kf, 1e-37f);
              p[j & 3] += c + j < hide ? 0.f : ex2(fminf(__fmul_rn(x[j], f) + lse[c + j], 0.f));
            }
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[s]);
          acc += (p[0] + p[1]) + (p[2] + p[3]);
          continue;
        }
#pragma unroll
        for (int c = 0; c < kSumCols; c += 32) {
          float x[32];
          tmem_ld_32cols(t_s + s * 256 + c, reinterpret_cast<uint32_t*>(x));
          tmem_ld_wait();
          if (c + 32 == kSumCols) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[s]);
          }
          if (rt >= clear) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 z = *reinterpret_cast<const float4*>(lse + c + j);
              fma2(x[j], x[j + 1], cf, z.x, z.y);
              fma2(x[j + 2], x[j + 3], cf, z.z, z.w);
              add2(p[0], p[1], ex2(x[j]), ex2(x[j + 1]));
              add2(p[2], p[3], ex2(x[j + 2]), ex2(x[j + 3]));
            }
          } else {
            const int64_t first = need - static_cast<int64_t>(rt) * kTileRows - part * kSumCols - c;
            const int hide =
                static_cast<int>(max(static_cast<int64_t>(0), min(first, static_cast<int64_t>(32))));
#pragma unroll
            for (int j = 0; j < 32; ++j)
              p[j & 3] += j < hide ? 0.f : ex2(fmaf(x[j], cf, lse[c + j]));
          }
        }
        acc += (p[0] + p[1]) + (p[2] + p[3]);
      }
      // ---- the columns' parts, then the other CTAs'
      sum_sync();
      if (part != 0) sum_s[threadIdx.x - 128] = acc;
      sum_sync();
      const size_t at = head() * a.weights_stride + key;
      const bool have = part == 0 && key < g.s.n;
      auto store = [&](float x) {
        if (have) a.weights_out[at] = (a.weights != nullptr ? a.weights[at] : 0.f) + x;
      };
      if (part == 0) {
#pragma unroll
        for (int x = 0; x < kSumParts - 1; ++x) acc += sum_s[128 * x + threadIdx.x];
      }
      // no rows: nothing has written these tiles; or the token's page is out of range
      if (g.s.m == 0 || kf == 0.f) acc = 0.f;
      if (g.lo == 0 && g.hi == g.units) {
        store(acc);
      } else {
        if (part == 0) __stcg(ws.sums + (2 * me + (g.lo == 0 ? 1 : 0)) * 128 + threadIdx.x, acc);
        const Shares shares(plan.total, plan.ctas);
        const uint32_t i0 = shares.of(g.item_base), i1 = shares.of(g.item_base + g.units - 1);
        sum_sync();
        if (threadIdx.x == 0) {
          __threadfence();
          uint32_t* cnt = ws.kcounters + head() * ws.key_tiles + g.kt;
          const bool last = atomicAdd(cnt, 1u) == static_cast<uint32_t>(i1 - i0);
          if (last) *cnt = 0u;
          __threadfence();
          *arrived = last ? 1u : 0u;
        }
        sum_sync();
        if (*arrived && part == 0) {
          float x = 0.f;
          for (uint32_t i = i0; i <= i1; ++i)
            x += __ldcg(ws.sums + (2 * i + (i == i0 ? 1 : 0)) * 128 + threadIdx.x);
          store(x);
        }
      }
    } while (advance(g, a, G));
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kSumWarps + 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

struct Layout {
  size_t plan, starts, order, base, pre, meta, token_meta, qf, row_qf, q_img, kv_img, counters,
      parts, lse2, kbase, kpre, kcounters, sums, total;
  int key_tiles, row_tiles;
};

Layout layout(int batch, int tokens, int max_new, int max_len, int heads, int kv_heads, int D,
              bool weights) {
  Layout l = {};
  const int G = heads / kv_heads;
  const size_t bh = static_cast<size_t>(batch) * kv_heads;
  l.key_tiles = (max_len + kTileKeys - 1) / kTileKeys;
  l.row_tiles = static_cast<int>((static_cast<int64_t>(max_new) * G + kTileRows - 1) / kTileRows);
  size_t at = kKv4CounterBytes;  // left alone: they stay zero for calls of few rows
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  l.counters = take(bh * l.row_tiles * 2 * 4);
  if (weights) l.kcounters = take(bh * l.key_tiles * 4);
  l.plan = take(2 * sizeof(Plan));
  l.starts = take(2 * static_cast<size_t>(device_sm_count()) * sizeof(Start));
  l.order = take(kOrdered * sizeof(Start));
  l.base = take((static_cast<size_t>(batch) + 1) * 4);
  l.pre = take(static_cast<size_t>(batch) * (l.row_tiles + 1) * 4);
  l.meta = take(bh * l.key_tiles * sizeof(KeyMeta));
  l.token_meta = take(bh * l.key_tiles * kTileKeys * sizeof(TokenMeta));
  l.qf = take(bh * l.row_tiles * 4);
  l.row_qf = take(bh * l.row_tiles * kTileRows * 4);
  l.q_img = take(bh * l.row_tiles * kTileRows * (D + 16) * 2);
  l.kv_img = take(bh * l.key_tiles * kTileKeys * (2 * D + 16) * 2);
  l.parts = take(static_cast<size_t>(device_sm_count()) * 4 * (D + 2) * 128 * 4);
  if (weights) {
    l.lse2 = take(bh * l.row_tiles * kTileRows * 4);
    l.kbase = take((static_cast<size_t>(batch) + 1) * 4);
    l.kpre = take(static_cast<size_t>(batch) * (l.key_tiles + 1) * 4);
    l.sums = take(static_cast<size_t>(device_sm_count()) * 2 * 128 * 4);
  }
  l.total = at;
  return l;
}

template <int D, int NG>
cudaError_t run(const Kv4AttentionArgs& a, cudaStream_t stream) {
  const bool weights = a.weights_out != nullptr;
  const Layout l = layout(a.c.batch, a.tokens, a.max_new, a.max_len, a.heads, a.c.kv_heads, D,
                          weights);
  uint8_t* w = a.workspace;
  PromptWs ws;
  ws.plan = reinterpret_cast<Plan*>(w + l.plan);
  ws.starts = reinterpret_cast<Start*>(w + l.starts);
  ws.order = reinterpret_cast<Start*>(w + l.order);
  ws.base = reinterpret_cast<uint32_t*>(w + l.base);
  ws.pre = reinterpret_cast<int32_t*>(w + l.pre);
  ws.meta = reinterpret_cast<KeyMeta*>(w + l.meta);
  ws.tokens = reinterpret_cast<TokenMeta*>(w + l.token_meta);
  ws.qf = reinterpret_cast<float*>(w + l.qf);
  ws.row_qf = reinterpret_cast<float*>(w + l.row_qf);
  ws.q_img = w + l.q_img;
  ws.kv_img = w + l.kv_img;
  ws.counters = reinterpret_cast<uint32_t*>(w + l.counters);
  ws.parts = reinterpret_cast<float*>(w + l.parts);
  ws.lse2 = weights ? reinterpret_cast<float*>(w + l.lse2) : nullptr;
  ws.kbase = weights ? reinterpret_cast<uint32_t*>(w + l.kbase) : nullptr;
  ws.kpre = reinterpret_cast<int32_t*>(w + l.kpre);
  ws.kcounters = reinterpret_cast<uint32_t*>(w + l.kcounters);
  ws.sums = reinterpret_cast<float*>(w + l.sums);
  ws.key_tiles = l.key_tiles;
  ws.row_tiles = l.row_tiles;
  const int64_t bh = static_cast<int64_t>(a.c.batch) * a.c.kv_heads;
  const int64_t units = bh * l.row_tiles * (l.key_tiles + kItemCost);
  if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid =
      static_cast<unsigned>(units < device_sm_count() ? units : device_sm_count());
  ws.grid = grid;
  const int64_t blocks = 2 + bh * (l.row_tiles + l.key_tiles);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_with_pdl(kv4_prompt_images_kernel<D, NG>,
                                  dim3(static_cast<unsigned>(blocks)), dim3(kImgThreads), 0, stream,
                                  a, ws);
  if (e != cudaSuccess) return e;
  auto kern = kv4_prompt_kernel<D>;
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), Smem<D>::alloc);
  if (e != cudaSuccess) return e;
  e = launch_with_pdl(kern, dim3(grid), dim3(kPromptThreads), Smem<D>::alloc, stream, a, ws);
  if (e != cudaSuccess || !weights) return e;
  auto wkern = kv4_prompt_weights_kernel<D>;
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(wkern), WeightSmem<D>::alloc);
  if (e != cudaSuccess) return e;
  return launch_with_pdl(wkern, dim3(grid), dim3(kWeightThreads), WeightSmem<D>::alloc, stream, a,
                         ws);
}

}  // namespace

size_t kv4_prompt_workspace(int batch, int tokens, int max_new, int max_len, int heads,
                            int kv_heads, int head_dim, bool weights) {
  return layout(batch, tokens, max_new, max_len, heads, kv_heads, head_dim, weights).total;
}

cudaError_t launch_kv4_prompt(const Kv4AttentionArgs& a, int head_dim, int group,
                              cudaStream_t stream) {
  if (head_dim == 128)
    return group == 128 ? run<128, 1>(a, stream)
           : group == 64 ? run<128, 2>(a, stream) : run<128, 4>(a, stream);
  return group == 64 ? run<64, 1>(a, stream) : run<64, 2>(a, stream);
}

}  // namespace w4k
