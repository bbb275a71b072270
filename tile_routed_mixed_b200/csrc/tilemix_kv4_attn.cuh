// Attention over the paged 4-bit cache (tilemix_kv4_attn).
//
// A unit of work is one (sequence, KV head, block of columns); a column is one
// query token of one of the KV head's query heads, and a block has 8 NB of
// them.  A unit's keys are cut into tiles of 32.  All tiles of all units, in
// order, are dealt out in equal contiguous ranges to the warps of the grid, so
// the split over a long axis and the balance of a ragged batch are the same
// thing.  A warp works alone: it streams its tiles through a ring of its own
// in shared memory (cp.async), with its own running maximum, sum and output,
// and meets the other warps of its CTA only once, at the end, where a thread
// goes through all of the CTA's partial states; units that CTAs share are
// finished by the last of theirs to arrive.  No warp waits for another CTA.
//
// Products.  The step reads each cached byte once; HBM brings the 4.2 to 4.6 KB
// of a tile to an SM in about 190 cycles.  What has to be short is the way from
// 4 bits to an operand of the matrix product:
//   - codes are stored as u = code + 8: a nibble in the low bits of an fp16
//     whose exponent field is that of 1024 makes it 1024 + u (one three-input
//     logic operation), and one packed addition leaves the code itself, an exact
//     integer; a nibble four bits up makes 1024 + 16 u, and the packed
//     multiply-add by 1/16 does as much.  Nine instructions for eight codes.
//     (Masked nibbles are also exact operands as they stand, as fp16
//     subnormals, at five instructions or eight.  But then 8 sum(P) has to come
//     off sums that are large against the result: over 16,000 keys a warp, with
//     the truncation in the products' sums, that cost a factor of three in O's
//     error; and at five instructions products are aligned by the subnormals'
//     exponent and lose six bits more.  A nibble in a byte is also the e4m3
//     number u 2^-9, at three instructions, but mma.sync on e4m3 is carried out
//     as conversions and fp16 products here: 380 us for 274, largest batch.)
//   - keys are the rows (M = 16) of the scores' product and channels those of
//     P V: S^T = K Q^T, O^T = V^T P^T, so no row is padding and the query columns
//     are the narrow side (N = 8).  (Queries as rows of S would save P's
//     transposition, but needs registers for zero rows: 390 us for 256.)
// Q is scaled per column by a power of two, so its largest magnitude is near
// 2^14 and every channel keeps at least 11 bits (fp16 has 5 of exponent,
// bf16 has 8) down to 2^-28 of it.  In bf16, whose K scales reach 2^125, K's
// codes enter as 2^-10 of themselves and Q's largest is near 2 (its 8 bits kept
// down to 2^-17 of it), so that no score before its factor passes fp32.  K's scales multiply the scores, V's the
// probabilities: P s_v is what is rounded to fp16 (11 bits).  A column's
// probabilities are 2^(score - r) with r = the largest score + log2 of the largest V scale (its
// power of two) - 5, so P s_v stays near 2^5 at the top, and r moves only when
// a score passes the old largest by 8 or a scale doubles: P s_v stays below
// 2^14, and fp32 holds the sums.  r cancels between O and the sum.  That serves
// scores below 2^22 and V scales within 2^-30 .. 2^40 that do not grow fourfold
// in keys that only some columns of a unit see.  A warp that meets anything else
// takes the unit's remaining tiles in a second, wide form of the tile: there each
// column goes by the V scales that it sees, takes bf16's largest and smallest times a
// power of two of its own, and large scores are taken against the largest before their
// rounding can matter.  (It costs plain calls what more code costs: 8 x 4096 19.0
// us for 18.6, a step 49.5 for 48.1; in one form, behind branches, 18.9 and 50.6.)
//
// Layouts.  With MMA fragments (rows g and g + 8, column pairs q4) a lane's
// operands of K are D / 32 words of a key's row, 16 (or 8) bytes together in
// the pool's order, and those of V 8 (or 4) bytes of four keys.  Row r of a
// block of 16 is key r ^ ((r >> 1) & 1): the four keys that a quarter of the
// lanes reads from V, and the two that eight lanes read from K, then fall
// into different banks (with V's 16-byte chunks exchanged by bit 2 of the key).
//
// Measured (B200; from a graph of calls over three caches in turn): 64 ragged
// sequences of up to 32768 tokens, 32/8 heads of 128, groups of 32: 1.22 GB in
// 256 to 272 us, 4.5 to 4.8 TB/s, 0.69 to 0.73 of the measured copy rate (267 to
// 292 us as single calls, in turn with a plain form).  What bounds it is a warp's
// own chain from load to product, with three warps a scheduler to overlap:
// 37 sequences of 16384 tokens take 696 instructions a tile, at full issue 174
// cycles of the SM's four schedulers and so less than the tile's bytes, but only
// 0.66 of the slots issue.  Of a warp's 4.5 cycles an instruction, 1 is its issue,
// 0.97 a fixed wait for the one before, 0.88 another ready warp's turn, 0.65 and
// 0.43 a busy pipe (ALU 0.51) or dispatch, 0.12 a load; DRAM 0.54 of nominal.  The
// arithmetic without the copies took 241 to 246 us, of which K's way to an operand
// is about 23, V's 36, the scaling and transposition of P 10, the exponentials 5;
// the rest is not attributed to single steps.  8 x 4096: 19 us; one sequence of
// 65536: 29.7 us, of 777: 10.7 us, of which 3.5 pass before the first tile is read.
// Included by tilemix_kv4.cu.
#pragma once

namespace tilemix {

constexpr int kAttnKeys = 32;  // keys of a tile

// Warps of a CTA (one CTA per SM), by column blocks.  Eight columns fit 168
// registers a thread; with 16 warps of 128 the largest batch is as fast (262 us,
// 259 with 12, 283 with 8), but a single short sequence has more states to combine
// (12.6 us, 11.5, 10.8).  Sixteen columns need 255.
template <int NB>
constexpr int kAttnWarps = NB == 1 ? 12 : 8;
constexpr int kAttnMaxCtas = 160;  // at least one per SM (148 on a B200)
// Tiles a CTA takes at least, while there are any (16: one sequence of 777 11.7 us
// for 10.5).
constexpr int kAttnMinTiles = 8;

namespace kv4 {

// 16 bytes from global to shared memory; off, a byte offset, is added to both.
template <int OFF_DST, int OFF_SRC>
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src),
               "n"(OFF_DST), "n"(OFF_SRC)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D[16x8] = A[16x16] * B[16x8], fp16 inputs, fp32 sums from zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// K's codes, in bf16 2^-10 of them.
template <bool DOWN>
__device__ __forceinline__ uint32_t k_low(uint32_t x) {
  if constexpr (!DOWN) return code_low(x);
  uint32_t y = or_1024(x, 0x000F000Fu);  // (1024 + u) 2^-10 - (1 + 2^-7)
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(y) : "r"(0x14001400u), "r"(0xBC08BC08u));
  return y;
}
template <bool DOWN>
__device__ __forceinline__ uint32_t k_high(uint32_t x) {
  if constexpr (!DOWN) return code_high(x);
  uint32_t y = or_1024(x, 0x00F000F0u);  // (1024 + 16 u) 2^-14 - (2^-4 + 2^-7)
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(y) : "r"(0x04000400u), "r"(0xAC80AC80u));
  return y;
}

// Larger magnitude-ordered half of two packed non-negative values (NaNs drop out).
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  } else {
    const __half2 m =
        __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float max_over_rows(float x) {  // over the lanes of a column pair
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_over_rows(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Powers of two that the largest V scale takes part in a column's reference with.
// Within kVPlain, references of any two partial states lie so near that no weight
// is lost, and sums of V within fp32.  Beyond (bf16 only) scales are taken times
// 2^-v_shift, to where 2^95 times 2^8 times the keys of a warp, and 2^-88 less 38 bits,
// are still fp32.
constexpr int kVPlainLow = -30, kVPlainHigh = 40;
template <bool BF16>
constexpr int kVLow = BF16 ? -90 : -60;  // (fp16's smallest is 2^-24: for zeros)
constexpr int kVHigh = 93;
constexpr int kVNone = -200;  // no V scale but zeros so far
// A V scale from v_lim = 2^(the power of the largest so far + 1) on moves the
// reference; this before the first.
constexpr float kVStart = 0x1.8p-59f;
__device__ __forceinline__ int exponent(float x) {  // -127 for zeros and subnormals
  return static_cast<int>(min(__float_as_uint(x) >> 23, 253u)) - 127;
}
__device__ __forceinline__ int power_of(float x) {  // of a largest scale
  return x > 0.f ? max(exponent(x), -126) : kVNone;
}
__device__ __forceinline__ float two_to(int e) {  // e in -126 .. 127
  return __int_as_float((e + 127) << 23);
}
__device__ __forceinline__ int v_shift(int top) {
  if (top == kVNone) return 0;
  return top > kVHigh ? top - kVHigh : min(top - kVLow<true>, 0);
}
// What the schedule needs to know about a sequence.
struct SeqWork {
  int len, queries, row0;  // keys, query tokens, first row of q
  int blocks, tiles;       // column blocks, key tiles of a unit
};
template <int NB>
__device__ __forceinline__ SeqWork seq_work(const Kv4AttnParams& p, int s) {
  SeqWork w;
  const int top = static_cast<int>(
      min(static_cast<long long>(p.max_pages) << p.pool.page_shift, 0x7fffff00LL));
  w.len = min(max(__ldg(p.seq_len + s), 0), top);
  if (p.granted && __ldg(p.granted + s) == 0) w.len = 0;  // its queries have no rows
  w.row0 = s;
  w.queries = 1;
  if (p.token_start) {
    w.row0 = __ldg(p.token_start + s);
    const long long n = static_cast<long long>(__ldg(p.token_start + s + 1)) - w.row0;
    w.queries = static_cast<int>(min(max(n, 0LL), static_cast<long long>(p.total_q)));
  }
  w.blocks = static_cast<int>((static_cast<unsigned>(w.queries) * p.group_q + 8 * NB - 1) / (8 * NB));
  w.tiles = max(1, (w.len + kAttnKeys - 1) / kAttnKeys);
  return w;
}
__device__ __forceinline__ long long seq_tiles(const Kv4AttnParams& p, const SeqWork& w) {
  return static_cast<long long>(p.pool.hk * w.blocks) * w.tiles;
}

// Column `col` of a unit's block: its row of q and its query head; false for
// padding (and for rows outside q).  total_q * hq < 2^31, so that columns fit.
template <int NB>
__device__ __forceinline__ bool column(const Kv4AttnParams& p, const SeqWork& w, int kv, int block,
                                       int col, int* token, int* row, int* head) {
  const unsigned c = block * (8u * NB) + col;
  const unsigned tok = c / p.group_q;
  *token = static_cast<int>(tok);
  *head = kv * p.group_q + static_cast<int>(c - tok * p.group_q);
  *row = w.row0 + *token;
  return *token < w.queries && *row >= 0 && *row < p.total_q;
}

// A unit as a warp meets it.
struct Unit {
  SeqWork w;
  int s, kv, block;
  int keys;  // keys that some column of the unit may see
};
// The unit after x, in the order sequence, KV head, block; there is one.
template <int NB>
__device__ __forceinline__ Unit unit_after(const Kv4AttnParams& p, Unit x) {
  int u = x.kv * x.w.blocks + x.block + 1;
  if (u == p.pool.hk * x.w.blocks) {
    u = 0;
    do {  // a sequence without queries has no unit
      x.s = min(x.s + 1, p.nseq - 1);
      x.w = seq_work<NB>(p, x.s);
    } while (x.w.blocks == 0 && x.s + 1 < p.nseq);
    x.w.blocks = max(x.w.blocks, 1);
  }
  x.kv = u / x.w.blocks;
  x.block = u - x.kv * x.w.blocks;
  const int last =
      min(static_cast<int>((x.block * (8u * NB) + 8u * NB - 1) / p.group_q), x.w.queries - 1);
  x.keys = max(0, x.w.len - x.w.queries + last + 1);
  return x;
}

// How the list of all tiles is cut: CTA c has tiles [begin(c), begin(c + 1)).
struct Cut {
  long long total, each;  // all tiles; total / ctas
  int ctas, rest;         // total % ctas
  long long a, b;         // this CTA's tiles: [a, b)
  __device__ __forceinline__ long long begin(int c) const {  // floor(c * total / ctas)
    return each * c + static_cast<unsigned>(c * rest) / static_cast<unsigned>(ctas);
  }
  // The CTA whose tiles hold tile x.
  __device__ __forceinline__ int holder(long long x) const {
    int c = static_cast<int>(min(x / each, static_cast<long long>(ctas - 1)));
    while (begin(c) > x) --c;
    return c;
  }
};

// A partial state (reference, sum and unnormalised output of every column of a
// unit): [columns][D] outputs, then [columns] references, then [columns] sums.
template <int D, int NB>
constexpr int kPartFloats = 8 * NB * (D + 2);

struct Part {
  long long first;  // the unit's first tile in the list of all tiles
  Unit unit;
  float* at;        // nullptr: none
};

// Counts an arrival (up to `last`, then from 0 again); what came before it is seen
// by those who arrive later.
__device__ __forceinline__ int arrive(unsigned* counter, int last) {
  unsigned was;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
               : "=r"(was)
               : "l"(counter), "r"(last)
               : "memory");
  return static_cast<int>(was);
}

// Four channels of a column while states are added up, in order.
struct Fold {
  float4 acc;
  float ref, sum;
  __device__ __forceinline__ void clear() {
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    ref = -INFINITY;
    sum = 0.f;
  }
  __device__ __forceinline__ void add(const float4& y, float r, float l) {
    const float to = fmaxf(ref, r), at = to == -INFINITY ? 0.f : to;
    const float wa = ptx::ex2(ref - at), wb = ptx::ex2(r - at);
    ref = to;
    sum = fmaf(sum, wa, l * wb);
    acc.x = fmaf(acc.x, wa, y.x * wb);
    acc.y = fmaf(acc.y, wa, y.y * wb);
    acc.z = fmaf(acc.z, wa, y.z * wb);
    acc.w = fmaf(acc.w, wa, y.w * wb);
  }
};

// Four channels of a finished column to O, and its LSE.
template <int D, int NB, bool BF16>
__device__ __forceinline__ void store_column(const Kv4AttnParams& p, const Unit& u, int col, int ch,
                                             const float4& acc, float ref, float sum) {
  int tok, row, hq;
  if (!column<NB>(p, u.w, u.kv, u.block, col, &tok, &row, &hq)) return;
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  *reinterpret_cast<uint2*>(p.o + ((static_cast<size_t>(row) * p.hq + hq) * D + ch) * 2) =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (ch == 0 && p.lse)
    p.lse[static_cast<size_t>(hq) * p.total_q + row] =
        sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace kv4

// A CTA's shared memory beside the rings.
template <int NB>
struct AttnShared {
  static constexpr int kWarps = kAttnWarps<NB>;
  kv4::Unit units_ahead[kWarps][8];  // from the one computed to the one fetched
  kv4::Part parts[2 * kWarps];
  const float* state[2 * kWarps];  // the partial states there are, in order
  kv4::Cut cuts[kWarps];  // each warp's: kept out of the registers meanwhile
  // first and last CTA of the unit that the CTA's first, and its last, tile is of
  int holders[2][2];
  int state_of[2 * kWarps];
  int last_here[2];  // states to combine, if this CTA is the last to arrive
};

template <int D, int GROUP, int NB>
struct AttnTile {
  static constexpr int kNg = D / GROUP;                 // scales per row
  static constexpr int kT = D / 32;                     // 32-channel chunks of a row
  static constexpr int kCodes = kAttnKeys * D / 2;      // bytes of K's (and V's) codes
  static constexpr int kScales = kAttnKeys * 2 * kNg;   // ... and scales
  static constexpr int kBytes = 2 * kCodes + 2 * kScales;
  static constexpr int kOffV = kCodes;
  static constexpr int kOffKs = 2 * kCodes;
  static constexpr int kOffVs = 2 * kCodes + kScales;
  // as many stages as fit beside the kernel's own, at most six
  static constexpr int kFit = (227 * 1024 - static_cast<int>(sizeof(AttnShared<NB>))) / (kAttnWarps<NB> * kBytes);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static_assert(kStages * kBytes * kAttnWarps<NB> + sizeof(AttnShared<NB>) <= 227 * 1024, "shared memory");
  static_assert(kStages >= 3, "ring too short");
  static_assert(kStages * kBytes >= 8 * NB * (D + 2) * 4, "a partial state fits a warp's ring");
};

// What a warp keeps of each column beside its state once it is in the wide form.
template <int NB>
struct Beyond {
  bool against;      // scores are taken against raw
  int power[NB][2];  // power of two of the largest V scale that the column has seen
  int shift[NB][2];  // V's scales are taken times 2^-shift
  float raw[NB][2];  // the largest score, before cs
};

template <int D, int GROUP, int NB, bool BF16>
__global__ void __launch_bounds__(32 * kAttnWarps<NB>, 1)
    kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  using Tile = AttnTile<D, GROUP, NB>;
  constexpr int kWarps = kAttnWarps<NB>, kThreads = 32 * kWarps;
  constexpr int kNg = Tile::kNg, kT = Tile::kT, kStages = Tile::kStages;
  constexpr int kCols = 8 * NB;
  constexpr int kTg = kT / kNg;  // chunks per scale group
  static_assert(2 * kWarps <= 32, "runs are found with one ballot");
  extern __shared__ __align__(128) uint8_t attn_smem[];
  __shared__ AttnShared<NB> shared;
  auto& units_ahead = shared.units_ahead;
  auto& parts = shared.parts;
  auto& state = shared.state;
  auto& cuts = shared.cuts;
  auto& holders = shared.holders;
  auto& state_of = shared.state_of;
  auto& last_here = shared.last_here;
  static_assert(kStages < 8, "a tile ahead may be a unit ahead");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;

  // ---- the schedule, by every warp for itself: this warp's tiles [wa, wb) ----
  long long wa, wb;
  int seq;
  long long off;  // of tile wa within sequence seq's tiles
  kv4::SeqWork seq_at;
  {
    kv4::Cut cut;
    const int per = (p.nseq + 31) / 32;
    const int s0 = min(p.nseq, lane * per), s1 = min(p.nseq, s0 + per);
    long long mine = 0;
    int units = 0, shortest = 0x7fffffff, longest = 0;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const kv4::SeqWork w = kv4::seq_work<NB>(p, s);
      mine += kv4::seq_tiles(p, w);
      units = min(units + p.pool.hk * w.blocks, 1 << 20);  // all that matters: fewer than CTAs?
      if (w.blocks > 0) shortest = min(shortest, w.tiles), longest = max(longest, w.tiles);
    }
    long long upto = mine;
#pragma unroll
    for (int by = 1; by < 32; by <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, upto, by);
      if (lane >= by) upto += up;
    }
    units = __reduce_add_sync(0xffffffffu, units);
    cut.total = __shfl_sync(0xffffffffu, upto, 31);
    // CTAs that take part: all, while each gets a few tiles.  Units of one length
    // are better cut at their own ends, the same number of CTAs for each, if that
    // leaves no more than a seventh of the CTAs idle: no CTA then has parts of two
    // units (8 x 4096, 24/8 heads: 18.6 us on 128 CTAs, 20.3 on 148; twelve ragged
    // sequences of 35 columns: 53 us on all, 76 on a number for each unit).
    const int some = static_cast<int>(min(cut.total, 1LL << 30));
    cut.ctas = min(static_cast<int>(gridDim.x), max(units, some / kAttnMinTiles));
    if (units <= cut.ctas && units > 0 &&
        __reduce_min_sync(0xffffffffu, shortest) == __reduce_max_sync(0xffffffffu, longest)) {
      const int aligned = units * max(1, min(some / (units * kAttnMinTiles), cut.ctas / units));
      if (aligned * 7 >= cut.ctas * 6) cut.ctas = aligned;
    }
    if (static_cast<int>(blockIdx.x) >= cut.ctas || cut.total == 0) return;
    if (cut.total <= 0x7fffffffLL) {
      cut.each = static_cast<unsigned>(cut.total) / static_cast<unsigned>(cut.ctas);
    } else {
      cut.each = cut.total / cut.ctas;
    }
    cut.rest = static_cast<int>(cut.total - cut.each * cut.ctas);
    cut.a = cut.begin(blockIdx.x);
    cut.b = cut.begin(blockIdx.x + 1);
    wa = cut.a + (cut.b - cut.a) * warp / kWarps;
    wb = cut.a + (cut.b - cut.a) * (warp + 1) / kWarps;
    if (lane == 0) cuts[warp] = cut;
    // the sequence that holds tile wa: the lane's share, then one by one
    const uint32_t from = __ballot_sync(0xffffffffu, upto - mine <= wa);
    const int at = 31 - __clz(from);
    seq = min(at * per, p.nseq - 1);
    off = wa - __shfl_sync(0xffffffffu, upto - mine, at);
#pragma unroll 1
    for (int i = 1;; ++i) {
      seq_at = kv4::seq_work<NB>(p, seq);
      const long long n = kv4::seq_tiles(p, seq_at);
      if (off < n || i >= per || seq + 1 >= p.nseq) break;
      off -= n;
      ++seq;
    }
    seq_at.blocks = max(seq_at.blocks, 1);
  }
  if (lane < 2) parts[2 * warp + lane].at = nullptr;
  __syncwarp();

  // ---- this warp's tiles ----
  if (wa < wb) {
    uint8_t* ring = attn_smem + warp * (kStages * Tile::kBytes);
    kv4::Unit* ahead = units_ahead[warp];
    // tile wa: in unit u of sequence seq, whose predecessor stands in the list
    const int u = off <= 0x7fffffffLL
                      ? static_cast<int>(static_cast<unsigned>(off) / static_cast<unsigned>(seq_at.tiles))
                      : static_cast<int>(off / seq_at.tiles);
    const int t_first = static_cast<int>(off - static_cast<long long>(u) * seq_at.tiles);
    if (lane == 0) ahead[7] = {seq_at, seq, 0, u - 1, 0};
    __syncwarp();
    int in_t = 0, in_tiles = 0, in_keys = 0, in_kv = 0, in_units = 0;
    const int32_t* in_table = nullptr;
    const int page_sh = p.pool.page_shift, page_1 = (1 << page_sh) - 1;
    const int count = static_cast<int>(wb - wa);
    int issued = 0;
    // Copies of a tile, 16 bytes a lane: each half of K's and V's codes (16 keys,
    // within one page) is D / 64 rounds of the warp, all four parts of the
    // scales together are one.  V's 16-byte chunks of a 64-byte row are exchanged by
    // bit 2 of the key.
    const uint32_t dst0 = ptx::smem_addr(ring) + lane * 16;
    const uint32_t dstv0 = ptx::smem_addr(ring) + Tile::kOffV +
                           (D == 128 ? (lane * 16) ^ ((lane & 16) << 1) : lane * 16);
    const int64_t v_minus_k = p.pool.v_codes - p.pool.k_codes;
    const int sc_half = (lane / (2 * kNg)) & 1;
    const uint8_t* sc_src = (lane < 4 * kNg ? p.pool.k_scale : p.pool.v_scale) + (lane % (2 * kNg)) * 16;
    int page_next = 0;
    // Tiles are fetched in runs: tiles of one page, or (run_reads false) tiles
    // that no column sees, which are passed over.  A run's sources: this lane's
    // 16 bytes of the first and second sixteen keys of K, and of the scales.
    int run = 0;
    bool run_reads = false;
    const uint8_t *k_lo = nullptr, *k_hi = nullptr, *sc = nullptr;
    const auto next_run = [&]() {
      if (in_t == in_tiles) {
        const kv4::Unit x = kv4::unit_after<NB>(p, ahead[(in_units - 1) & 7]);
        if (lane == 0) ahead[in_units & 7] = x;
        __syncwarp();
        in_t = in_units == 0 ? t_first : 0;
        ++in_units;
        in_keys = x.keys, in_tiles = x.w.tiles, in_kv = x.kv;
        in_table = p.block_table + static_cast<size_t>(x.s) * p.max_pages;
        if (in_t * kAttnKeys < in_keys) page_next = __ldg(in_table + ((in_t * kAttnKeys) >> page_sh));
      }
      const int key = in_t * kAttnKeys;
      run_reads = key < in_keys;
      if (!run_reads) {
        run = in_tiles - in_t;
        in_t = in_tiles;
      } else {
        // a page outside the pool is reported, and page 0 read in its place
        int lo = page_next, hi = page_next;
        if (page_sh == 4) {
          // two pages; the second sixteen may have no key to see: then the first again
          run = 1;
          if (key + 16 < in_keys) hi = __ldg(in_table + (key >> 4) + 1);
        } else {
          run = min((page_1 + 1 - (key & page_1)) / kAttnKeys, (in_keys - key + kAttnKeys - 1) / kAttnKeys);
        }
        if (static_cast<unsigned>(lo) >= static_cast<unsigned>(p.pool.num_pages) ||
            static_cast<unsigned>(hi) >= static_cast<unsigned>(p.pool.num_pages)) {
          atomicOr(&g_kv4_status, kStatusBadPages);
          lo = hi = 0;
        }
        const size_t row_lo = ((static_cast<size_t>(lo) * p.pool.hk + in_kv) << page_sh) + (key & page_1);
        const size_t row_hi = page_sh == 4 ? (static_cast<size_t>(hi) * p.pool.hk + in_kv) << 4 : row_lo + 16;
        k_lo = p.pool.k_codes + row_lo * (D / 2) + lane * 16;
        k_hi = p.pool.k_codes + row_hi * (D / 2) + lane * 16;
        sc = sc_src + (sc_half ? row_hi : row_lo) * (2 * kNg);
        in_t += run;
        const int then = in_t * kAttnKeys;
        if (then < in_keys) page_next = __ldg(in_table + (then >> page_sh));
      }
    };

    // Fetches the next tile into `stage`.
    const auto issue = [&](int stage) {
      if (issued < count) {
        ++issued;
        if (run == 0) next_run();
        --run;
        if (run_reads) {
          const uint32_t dst = dst0 + stage * Tile::kBytes, dstv = dstv0 + stage * Tile::kBytes;
          kv4::cp16<0, 0>(dst, k_lo);
          kv4::cp16<0, 0>(dstv, k_lo + v_minus_k);
          kv4::cp16<8 * D, 0>(dst, k_hi);
          kv4::cp16<8 * D, 0>(dstv, k_hi + v_minus_k);
          if constexpr (D == 128) {
            kv4::cp16<512, 512>(dst, k_lo);
            kv4::cp16<512, 512>(dstv, k_lo + v_minus_k);
            kv4::cp16<8 * D + 512, 512>(dst, k_hi);
            kv4::cp16<8 * D + 512, 512>(dstv, k_hi + v_minus_k);
          }
          // lanes: K's scales (two halves), then V's, in the order of the ring
          if (lane < 8 * kNg) kv4::cp16<Tile::kOffKs, 0>(dst, sc);
          k_lo += kAttnKeys * (D / 2);
          k_hi += kAttnKeys * (D / 2);
          sc += kAttnKeys * (2 * kNg);
        }
      }
      kv4::cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    int stage = 0;
    int left = count;
    int units_done = 0;
    long long unit_first = wa - t_first;
    // rows of a block of 16 that this lane reads: keys of rows g, 2 q4, 2 q4 + 1
    const int key_g = g ^ ((g >> 1) & 1);
    const int key_e0 = (2 * q4) ^ (q4 & 1), key_e1 = (2 * q4 + 1) ^ (q4 & 1);
    const int k_at = key_g * (D / 2) + q4 * (D / 8);
    const int v_in = D == 128 ? (((g >> 1) ^ ((q4 >> 1) << 1)) << 4) + (g & 1) * 8 : g * 4;
    const int v_at0 = Tile::kOffV + key_e0 * (D / 2) + v_in;
    const int v_at1 = Tile::kOffV + key_e1 * (D / 2) + v_in;
    const int sc_at = Tile::kOffKs + key_g * (2 * kNg);

#pragma unroll 1
    while (left > 0) {
      // ---- a unit: its queries ----
      const kv4::Unit& cur = ahead[units_done & 7];
      const int t0 = units_done == 0 ? t_first : 0, keys = cur.keys;
      const int n = max(1, min(left, cur.w.tiles - t0));  // (1: always onwards)
      const bool whole = t0 == 0 && n == cur.w.tiles;
      const bool head = !whole && n < left;  // more tiles of this warp follow
      // who else holds the CTA's first and last unit, found while loads are on the way
      if (lane == 0) {
        const kv4::Cut& cut = cuts[warp];
        for (int i = 0; i < 2; ++i)
          if (i == 0 ? wa == cut.a && units_done == 0 : wb == cut.b && n == left) {
            holders[i][0] = cut.holder(unit_first);
            holders[i][1] = cut.holder(unit_first + cur.w.tiles - 1);
          }
      }
      uint32_t qf[NB][kT][4];
      float cs[NB][2];  // scale of a column's scores, log2 units
      int lim[NB][2];  // keys that each column sees
      const int seen0 = cur.w.len - cur.w.queries + 1;  // ... of query token 0
      const int min_lim =
          min(seen0 + static_cast<int>(static_cast<unsigned>(cur.block) * kCols / p.group_q), cur.w.len);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        int tok, row, hq;
        const bool on = kv4::column<NB>(p, cur.w, cur.kv, cur.block, 8 * nb + g, &tok, &row, &hq);
        const uint8_t* src = p.q + (static_cast<size_t>(on ? row : 0) * p.hq + (on ? hq : 0)) * (2 * D);
        uint4 x[kT];
        uint32_t am = 0;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          x[t] = make_uint4(0u, 0u, 0u, 0u);
          if (on) x[t] = __ldg(reinterpret_cast<const uint4*>(src + 16 * (4 * t + q4)));
          am = max(am, kv4::absmax_bits(x[t]));
        }
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // f = 2^(14 - exponent of the largest magnitude) (bf16: 2^(1 - exponent), but
        // from 2^61 on, where the score's factor would pass fp32), 1 for zeros,
        // infinities, NaN
        const uint32_t ex = __float_as_uint(kv4::unpack1<BF16>(am)) >> 23;
        const uint32_t fe = (am == 0 || am >= kv4::kInfBits<BF16>) ? 127u
                            : min((BF16 && ex < 188u ? 255u : 268u) - ex, 253u);
        const float f = __uint_as_float(fe << 23);
        const float inv_f = __uint_as_float((254u - fe) << 23);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const float2 c01 = kv4::unpack2<BF16>(x[t].x), c23 = kv4::unpack2<BF16>(x[t].y);
          const float2 c45 = kv4::unpack2<BF16>(x[t].z), c67 = kv4::unpack2<BF16>(x[t].w);
          qf[nb][t][0] = kv4::pack2<false>(c01.x * f, c45.x * f);
          qf[nb][t][1] = kv4::pack2<false>(c23.x * f, c67.x * f);
          qf[nb][t][2] = kv4::pack2<false>(c01.y * f, c45.y * f);
          qf[nb][t][3] = kv4::pack2<false>(c23.y * f, c67.y * f);
        }
        const float unit = (BF16 ? inv_f * 0x1p10f : inv_f) * p.scale_log2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int from = (2 * q4 + j) * 4;  // a lane of that column
          cs[nb][j] = __shfl_sync(0xffffffffu, unit, from);
          const int tk = __shfl_sync(0xffffffffu, tok, from);
          lim[nb][j] = tk < cur.w.queries ? seen0 + tk : cur.w.len;
        }
      }

      // ---- its running state ----
      float o[kT][2][NB][4];
      // per column: the reference r of its probabilities 2^(score - r), the score
      // that moves it, their sum; per unit: the V scale that moves it
      float r[NB][2], mv[NB][2], l[NB][2];
      float v_lim = kv4::kVStart;
      Beyond<NB> far = {};
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[t][i][nb][c] = 0.f;
        mv[nb][0] = mv[nb][1] = -INFINITY;
        r[nb][0] = r[nb][1] = 0.f;
        l[nb][0] = l[nb][1] = 0.f;
      }

      const uint8_t* st = nullptr;
      const auto next_tile = [&]() {
        kv4::cp_wait<kStages - 2>();
        __syncwarp();  // this tile is here for all lanes, and the last one is read
        issue(stage == 0 ? kStages - 1 : stage - 1);
        st = ring + stage * Tile::kBytes;
        stage = stage == kStages - 1 ? 0 : stage + 1;
      };

      const auto row_scale = [](const uint32_t (&x)[(kNg + 1) / 2]) {  // the largest of a row
        const float2 f = kv4::unpack2<BF16>(kNg == 4 ? kv4::max2<BF16>(x[0], x[(kNg - 1) / 2]) : x[0]);
        return fmaxf(f.x, f.y);
      };

      // A tile's keys into the state.  Plain, it stops (false, the state as it was)
      // where that would lose bits; `wide` is the form for all that hardly a tile
      // needs, which runs from there to the unit's end.
      const auto tile = [&](auto wide, int key0) -> bool {
        constexpr bool kWide = decltype(wide)::value;
        // scores, to be scaled by cs
        float s[2][NB][4];
        uint32_t vsc[2][2][(kNg + 1) / 2];  // V's scales of rows g and g + 8
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          uint32_t k0[kT], k1[kT];
          const uint8_t* kr = st + k_at + 16 * mb * (D / 2);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(kr);
            const uint4 y = *reinterpret_cast<const uint4*>(kr + 8 * (D / 2));
            k0[0] = x.x, k0[1] = x.y, k0[2] = x.z, k0[3] = x.w;
            k1[0] = y.x, k1[1] = y.y, k1[2] = y.z, k1[3] = y.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(kr);
            const uint2 y = *reinterpret_cast<const uint2*>(kr + 8 * (D / 2));
            k0[0] = x.x, k0[1] = x.y;
            k1[0] = y.x, k1[1] = y.y;
          }
          uint32_t ksc[2][(kNg + 1) / 2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* kp = st + sc_at + (16 * mb + 8 * h) * (2 * kNg);
            const uint8_t* vp = kp + Tile::kScales;
            if constexpr (kNg == 4) {
              const uint2 x = *reinterpret_cast<const uint2*>(kp), y = *reinterpret_cast<const uint2*>(vp);
              ksc[h][0] = x.x, ksc[h][1] = x.y;
              vsc[mb][h][0] = y.x, vsc[mb][h][1] = y.y;
            } else if constexpr (kNg == 2) {
              ksc[h][0] = *reinterpret_cast<const uint32_t*>(kp);
              vsc[mb][h][0] = *reinterpret_cast<const uint32_t*>(vp);
            } else {
              ksc[h][0] = *reinterpret_cast<const unsigned short*>(kp);
              vsc[mb][h][0] = *reinterpret_cast<const unsigned short*>(vp);
            }
          }
#pragma unroll
          for (int i = 0; i < kNg; ++i) {
            float acc[NB][4];
#pragma unroll
            for (int t = i * kTg; t < (i + 1) * kTg; ++t) {
              const uint32_t x = k0[t], y = k1[t], xh = x >> 8, yh = y >> 8;
              const uint32_t ev[4] = {kv4::k_low<BF16>(x), kv4::k_low<BF16>(y), kv4::k_low<BF16>(xh),
                                      kv4::k_low<BF16>(yh)};
              const uint32_t od[4] = {kv4::k_high<BF16>(x), kv4::k_high<BF16>(y), kv4::k_high<BF16>(xh),
                                      kv4::k_high<BF16>(yh)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                if (t == i * kTg)
                  kv4::mma_f16_first(acc[nb], ev, qf[nb][t][0], qf[nb][t][1]);
                else
                  dec::mma_f16(acc[nb], ev, qf[nb][t][0], qf[nb][t][1]);
                dec::mma_f16(acc[nb], od, qf[nb][t][2], qf[nb][t][3]);
              }
            }
            const float2 f0 = kv4::unpack2<BF16>(ksc[0][i / 2]), f1 = kv4::unpack2<BF16>(ksc[1][i / 2]);
            const float a0 = (i & 1) ? f0.y : f0.x, a1 = (i & 1) ? f1.y : f1.x;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                s[mb][nb][j] = i == 0 ? acc[nb][j] * a0 : fmaf(acc[nb][j], a0, s[mb][nb][j]);
                s[mb][nb][2 + j] =
                    i == 0 ? acc[nb][2 + j] * a1 : fmaf(acc[nb][2 + j], a1, s[mb][nb][2 + j]);
              }
          }
        }
        if (key0 + kAttnKeys > min_lim) {
          // keys that a column does not see; rows past the cache hold whatever
          // the ring held, so their V scales go too
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = key0 + 16 * mb + 8 * h + key_g;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (key >= lim[nb][j]) s[mb][nb][2 * h + j] = -INFINITY;
              if (key >= keys) {
#pragma unroll
                for (int i = 0; i < (kNg + 1) / 2; ++i) vsc[mb][h][i] = 0u;
              }
            }
          // A NaN among V's scales of keys that only some columns see: the masked
          // ones' zero probabilities would carry it on.  It goes to the outputs of
          // the columns that do see its key, and out of the product.
          bool odd_one = false;
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < (kNg + 1) / 2; ++i) {
                const float2 f = kv4::unpack2<BF16>(vsc[mb][h][i]);
                odd_one |= (isnan(f.x) || isnan(f.y)) && key0 + 16 * mb + 8 * h + key_g >= min_lim;
              }
          if (__any_sync(0xffffffffu, odd_one)) {
#pragma unroll
            for (int i = 0; i < kNg; ++i) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  bool hit = false;
#pragma unroll
                  for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const int key = key0 + 16 * mb + 8 * h + key_g;
                      const float2 f = kv4::unpack2<BF16>(vsc[mb][h][i / 2]);
                      hit |= isnan((i & 1) ? f.y : f.x) && key >= min_lim && key < lim[nb][j];
                    }
                  // the lanes that hold the same columns
                  if (__ballot_sync(0xffffffffu, hit) & (0x11111111u << q4)) {
#pragma unroll
                    for (int t = i * kTg; t < (i + 1) * kTg; ++t)
#pragma unroll
                      for (int x = 0; x < 2; ++x)
                        o[t][x][nb][j] = o[t][x][nb][2 + j] = __int_as_float(0x7fffffff);
                  }
                }
            }
#pragma unroll
            for (int mb = 0; mb < 2; ++mb)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (key0 + 16 * mb + 8 * h + key_g >= min_lim) {
#pragma unroll
                  for (int i = 0; i < (kNg + 1) / 2; ++i) {
                    const float2 f = kv4::unpack2<BF16>(vsc[mb][h][i]);
                    vsc[mb][h][i] &= (isnan(f.x) ? 0u : 0xffffu) | (isnan(f.y) ? 0u : 0xffff0000u);
                  }
                }
          }
        }

        // running maximum, and the power of two of V's scales
        float mx[NB][2];
        bool moved = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mx[nb][j] = cs[nb][j] * fmaxf(fmaxf(s[0][nb][j], s[0][nb][2 + j]),
                                          fmaxf(s[1][nb][j], s[1][nb][2 + j]));
            moved |= mx[nb][j] > mv[nb][j];
          }
        uint32_t vm = vsc[0][0][0];
#pragma unroll
        for (int x = 1; x < 4 * ((kNg + 1) / 2); ++x)
          vm = kv4::max2<BF16>(vm, vsc[x & 1][(x >> 1) & 1][x >> 2]);
        const float2 vm2 = kv4::unpack2<BF16>(vm);  // (one scale per row: the upper half is zero)
        float vmax = fmaxf(vm2.x, vm2.y);
        moved |= kWide || !(vmax < v_lim);
        if (__any_sync(0xffffffffu, moved)) {
          vmax = kv4::max_over_rows(vmax);
          float lg[NB][2];
          if constexpr (!kWide) {
            const int power = max(kv4::exponent(v_lim) - 1, kv4::exponent(vmax));
            bool stop = BF16 && (power < kv4::kVPlainLow || power > kv4::kVPlainHigh);
            // (scores from 2^22 on: no room for r's offset in their last bits, and a
            // fused score - r keeps bits that the maximum has lost)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                stop |= fabsf(mx[nb][j]) >= 0x1p22f && mx[nb][j] != -INFINITY;
            if (key0 + kAttnKeys > min_lim && min_lim < keys && vmax >= 2.0f * v_lim) {
              // keys that not all columns see, with scales four times all that they do
              float all = 0.f;
#pragma unroll
              for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (key0 + 16 * mb + 8 * h + key_g < max(min_lim, key0 + 1))
                    all = fmaxf(all, row_scale(vsc[mb][h]));
              stop |= vmax >= 4.0f * kv4::max_over_rows(all);
            }
            if (__any_sync(0xffffffffu, stop)) return false;
            v_lim = kv4::two_to(power + 1);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) lg[nb][0] = lg[nb][1] = static_cast<float>(power);
          } else {
            bool large = far.against;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int j = 0; j < 2; ++j) large |= fabsf(mx[nb][j]) >= 0x1p22f && mx[nb][j] != -INFINITY;
            const bool was_against = far.against, against = __any_sync(0xffffffffu, large);
            if (against) {
              // Scores, and what is there already, against the largest score (before
              // cs) first of all.
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const bool first = mv[nb][j] == -INFINITY;
                  const float before =
                      first ? -INFINITY : was_against ? far.raw[nb][j] : __fdividef(mv[nb][j] - 8.0f, cs[nb][j]);
                  const float t = fmaxf(before, kv4::max_over_rows(fmaxf(fmaxf(s[0][nb][j], s[0][nb][2 + j]),
                                                                         fmaxf(s[1][nb][j], s[1][nb][2 + j]))));
                  far.raw[nb][j] = t;
                  if (t != -INFINITY) {
                    if (!first) {
                      r[nb][j] = was_against ? (before - t) * cs[nb][j] : fmaf(-t, cs[nb][j], r[nb][j]);
                      mv[nb][j] = 8.0f;
                    }
                    mx[nb][j] = -INFINITY;
#pragma unroll
                    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                      for (int h = 0; h < 2; ++h) {
                        s[mb][nb][2 * h + j] -= t;
                        mx[nb][j] = fmaxf(mx[nb][j], cs[nb][j] * s[mb][nb][2 * h + j]);
                      }
                  }
                }
            }
            // Each column goes by the V scales that it does see, so that a later token's
            // cost an earlier query no bits.
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float seen = 0.f;
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (key0 + 16 * mb + 8 * h + key_g < lim[nb][j]) seen = fmaxf(seen, row_scale(vsc[mb][h]));
                const int power = max(far.power[nb][j], kv4::power_of(kv4::max_over_rows(seen)));
                // (against: probabilities are at most one, V's scales are taken to near 2^5)
                const int shift = against ? (power == kv4::kVNone ? 0 : max(power - 5, -126))
                                          : BF16 ? kv4::v_shift(power) : 0;
                const int at0 = max(far.power[nb][j] - far.shift[nb][j], kv4::kVLow<BF16>);
                const int at = against ? 5 : max(power - shift, kv4::kVLow<BF16>);
                lg[nb][j] = static_cast<float>(at);
                // the state in units of the new shift, and, where the reference jumps, 2^64
                // lower (one factor could lie below fp32's range)
                const int jump = BF16 && !against && at - at0 > 70 ? 64 : 0;
                const float fo = kv4::two_to(min(max(far.shift[nb][j] - shift - jump, -126), 126));
                l[nb][j] *= kv4::two_to(-jump);
                r[nb][j] += static_cast<float>(jump);
#pragma unroll
                for (int t = 0; t < kT; ++t)
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    o[t][i][nb][j] *= fo;
                    o[t][i][nb][2 + j] *= fo;
                  }
                far.power[nb][j] = power, far.shift[nb][j] = shift;
              }
            far.against = against;
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // largest score so far; -infinity while no key was seen
              const float top_s = fmaxf(mv[nb][j] - 8.0f, kv4::max_over_rows(mx[nb][j]));
              const float to = top_s == -INFINITY ? r[nb][j] : top_s + lg[nb][j] - 5.0f;
              const float ao = mv[nb][j] == -INFINITY ? 1.0f : ptx::ex2(r[nb][j] - to);
              r[nb][j] = to;
              mv[nb][j] = top_s + 8.0f;
              l[nb][j] *= ao;
#pragma unroll
              for (int t = 0; t < kT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  o[t][i][nb][j] *= ao;
                  o[t][i][nb][2 + j] *= ao;
                }
            }
        }

        // P and P V
        const auto scale_for = [&](float f, int nb, int j) {
          if constexpr (!kWide) return f;
          const float x = f * kv4::two_to(-far.shift[nb][j]);
          return x > 0x1p126f ? 0x1p126f : x;  // (finite where the column does not see it: 0 x)
        };
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              s[mb][nb][c] = ptx::ex2(fmaf(s[mb][nb][c], cs[nb][c & 1], -r[nb][c & 1]));
            l[nb][0] += s[mb][nb][0] + s[mb][nb][2];
            l[nb][1] += s[mb][nb][1] + s[mb][nb][3];
          }
          uint32_t v[4][kT / 2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint8_t* vr = st + ((e & 1) ? v_at1 : v_at0) + (16 * mb + 8 * (e >> 1)) * (D / 2);
            if constexpr (D == 128) {
              const uint2 x = *reinterpret_cast<const uint2*>(vr);
              v[e][0] = x.x, v[e][1] = x.y;
            } else {
              v[e][0] = *reinterpret_cast<const uint32_t*>(vr);
            }
          }
#pragma unroll
          for (int i = 0; i < kNg; ++i) {
            const float2 x0 = kv4::unpack2<BF16>(vsc[mb][0][i / 2]), x1 = kv4::unpack2<BF16>(vsc[mb][1][i / 2]);
            const float f0 = (i & 1) ? x0.y : x0.x, f1 = (i & 1) ? x1.y : x1.x;
            uint32_t pb[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              // (in the wide form each column takes V's scales its own way)
              const float f00 = scale_for(f0, nb, 0), f01 = scale_for(f0, nb, 1);
              const float f10 = scale_for(f1, nb, 0), f11 = scale_for(f1, nb, 1);
              pb[nb][0] = kv4::transpose8x8(kv4::pack2<false>(s[mb][nb][0] * f00, s[mb][nb][1] * f01));
              pb[nb][1] = kv4::transpose8x8(kv4::pack2<false>(s[mb][nb][2] * f10, s[mb][nb][3] * f11));
            }
#pragma unroll
            for (int t = i * kTg; t < (i + 1) * kTg; ++t) {
              // channels 32 t + 4 g + {0, 2} and {1, 3} of keys e0, e1 | e2, e3
              const uint32_t pick = (t & 1) ? 0x7632u : 0x5410u;
              const uint32_t x = __byte_perm(v[0][t / 2], v[1][t / 2], pick);
              const uint32_t y = __byte_perm(v[2][t / 2], v[3][t / 2], pick);
              const uint32_t xh = x >> 8, yh = y >> 8;
              const uint32_t ev[4] = {kv4::code_low(x), kv4::code_low(xh), kv4::code_low(y),
                                      kv4::code_low(yh)};
              const uint32_t od[4] = {kv4::code_high(x), kv4::code_high(xh), kv4::code_high(y),
                                      kv4::code_high(yh)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                dec::mma_f16(o[t][0][nb], ev, pb[nb][0], pb[nb][1]);
                dec::mma_f16(o[t][1][nb], od, pb[nb][0], pb[nb][1]);
              }
            }
          }
        }
        return true;
      };

      int it = 0;
      bool wide = false;
#pragma unroll 1
      for (; it < n && !wide; it += !wide) {
        next_tile();
        const int key0 = (t0 + it) * kAttnKeys;
        // (of a tile behind the last key nothing was fetched)
        wide = key0 < keys && !tile(std::false_type(), key0);
      }
      if (wide) {
        far.against = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            far.power[nb][j] = v_lim == kv4::kVStart ? kv4::kVNone : kv4::exponent(v_lim) - 1;
            far.shift[nb][j] = 0;
          }
#pragma unroll 1
        for (;;) {
          const int key0 = (t0 + it) * kAttnKeys;
          if (key0 < keys) tile(std::true_type(), key0);
          if (++it == n) break;
          next_tile();
        }
      }

      // ---- the unit's end: to the outputs, or a partial state ----
      float* part = nullptr;
      if (!whole) {
        // a warp's last tiles leave their state in its ring, which is done with
        // (every copy into it was waited for); an earlier unit's (one at most: the
        // warp's first) goes to the workspace
        part = head ? p.heads + static_cast<size_t>(blockIdx.x * kWarps + warp) * kv4::kPartFloats<D, NB>
                    : reinterpret_cast<float*>(ring);
        if (lane == 0)
          parts[2 * warp + (head ? 0 : 1)] = {unit_first, cur, part};
      }
      __syncwarp();
      if (wide) {
        // Its unit is the V scales' within kVPlain, else the nearer end.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // the power in the column's reference
            int lg = mv[nb][j] == -INFINITY ? 0 : __float2int_rn(r[nb][j] - mv[nb][j] + 13.0f);
            const int shift = far.shift[nb][j];
            int unit = min(max(lg + shift, kv4::kVPlainLow), kv4::kVPlainHigh);
            if (far.against) {
              // (the same for all, so that equal scores of two states weigh the same)
              lg = 5, unit = shift > 80 ? kv4::kVPlainHigh : 5;
              r[nb][j] = far.raw[nb][j] * cs[nb][j];
            }
            const float to_o = kv4::two_to(lg + shift - unit), to_l = kv4::two_to(lg - unit);
            l[nb][j] *= to_l;
            r[nb][j] += static_cast<float>(unit - lg);
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                o[t][i][nb][j] *= to_o;
                o[t][i][nb][2 + j] *= to_o;
              }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float lsum = kv4::sum_over_rows(l[nb][j]);
          const float ref = lsum == 0.f ? -INFINITY : r[nb][j];
          const int col = 8 * nb + 2 * q4 + j;
#pragma unroll
          for (int t = 0; t < kT; ++t) {
            const float4 x = make_float4(o[t][0][nb][j], o[t][1][nb][j], o[t][0][nb][2 + j],
                                         o[t][1][nb][2 + j]);
            const int ch = 32 * t + 4 * g;
            if (!whole)
              *reinterpret_cast<float4*>(part + col * D + ch) = x;
            else
              kv4::store_column<D, NB, BF16>(p, cur, col, ch, x, ref, lsum);
          }
          if (!whole && g == 0) {
            part[kCols * D + col] = ref;
            part[kCols * (D + 1) + col] = lsum;
          }
        }
      left -= n;
      unit_first += cur.w.tiles;
      ++units_done;
    }
  }

  // ---- the CTA's partial states; what other CTAs share goes on ----
  // States lie in the order of the tiles, so those of one unit are neighbours: a
  // run.  A thread has a column's four channels and goes through all states once,
  // four loads ahead; where a run ends, the unit is finished or, if other CTAs
  // have tiles of it too (the first and the last unit may be such), its state
  // is passed on.
  __syncthreads();
  constexpr int kItems = kCols * (D / 4);
  constexpr size_t kPart = kv4::kPartFloats<D, NB>;
  uint32_t here, starts;  // states there are; those that begin a run
  {
    const bool present = lane < 2 * kWarps && parts[lane].at != nullptr;
    here = __ballot_sync(0xffffffffu, present);
    const uint32_t before = here & ((1u << lane) - 1u);
    starts = __ballot_sync(
        0xffffffffu, present && (before == 0 || parts[31 - __clz(before)].first != parts[lane].first));
    const uint32_t after = here & (lane == 31 ? 0u : 0xffffffffu << (lane + 1));
    if (present) {  // (every warp writes the same)
      state[__popc(before)] = parts[lane].at;
      // its place in parts, and whether it ends its run
      state_of[__popc(before)] = lane | (after == 0 || (starts >> (__ffs(after) - 1) & 1u) ? 64 : 0);
    }
    __syncwarp();
  }
  if (here == 0) return;
  const long long a = cuts[warp].a, b = cuts[warp].b;
  const auto shared_unit = [&](const kv4::Part& u) {
    return u.first < a || u.first + u.unit.w.tiles > b;
  };
  const int ends[2] = {__ffs(starts) - 1, 31 - __clz(starts)};
  int n = __popc(here), n0 = 0;
  bool again = false;
  const int* span0 = nullptr;
  const int* span1 = nullptr;
#pragma unroll 1
  for (;;) {
    // first this CTA's states; then, of the two shared units (if this CTA is the
    // last of theirs to arrive), n0 and n - n0 CTAs' states
    const auto at = [&](int k) -> const float* {
      if (!again) return state[k];
      const int* const span = k < n0 ? span0 : span1;
      const int c = k < n0 ? k : k - n0;
      return p.parts + static_cast<size_t>(2 * (span[0] + c) + (c == 0 ? 1 : 0)) * kPart;
    };
#pragma unroll 1
    for (int x = tid; x < kItems; x += kThreads) {
      const int col = x / (D / 4), ch = 4 * (x % (D / 4));
      float4 y[4];
      float r[4], l[4];
      const auto fetch = [&](int k, int slot) {
        if (k < n) {
          const float* from = at(k);
          y[slot] = *reinterpret_cast<const float4*>(from + col * D + ch);
          r[slot] = from[kCols * D + col];
          l[slot] = from[kCols * (D + 1) + col];
        }
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) fetch(j, j);
      kv4::Fold f;
      f.clear();
#pragma unroll 1
      for (int k0 = 0; k0 < n; k0 += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = k0 + j;
          if (k >= n) break;
          f.add(y[j], r[j], l[j]);
          fetch(k + 4, j);
          const int of = again ? (k + 1 == n0 ? ends[0] | 64 : k + 1 == n ? ends[1] | 64 : 0) : state_of[k];
          if (of & 64) {
            const kv4::Part& u = parts[of & 63];
            if (again || !shared_unit(u)) {
              kv4::store_column<D, NB, BF16>(p, u.unit, col, ch, f.acc, f.ref, f.sum);
            } else {
              // to this CTA's first place (the unit began before its tiles) or second
              float* out = p.parts + (2 * static_cast<size_t>(blockIdx.x) + (u.first < a ? 0 : 1)) * kPart;
              *reinterpret_cast<float4*>(out + col * D + ch) = f.acc;
              if (ch == 0) {
                out[kCols * D + col] = f.ref;
                out[kCols * (D + 1) + col] = f.sum;
              }
            }
            f.clear();
          }
        }
      }
    }
    if (again) return;
    again = true;
    const bool shares0 = shared_unit(parts[ends[0]]);
    const bool shares1 = ends[1] != ends[0] && shared_unit(parts[ends[1]]);
    if (!shares0 && !shares1) return;
    span0 = holders[parts[ends[0]].first < a ? 0 : 1];
    span1 = holders[1];
    __syncthreads();
    if (lane == 0 && warp < 2) {
      int last = 0;
      if (warp == 0 ? shares0 : shares1) {
        const int* const span = warp == 0 ? span0 : span1;
        const int others = span[1] - span[0];
        // wraps to zero with the last arrival, so the array is zero again
        last = kv4::arrive(p.sync + span[0], others) == others ? others + 1 : 0;
      }
      last_here[warp] = last;
    }
    __syncthreads();
    n0 = last_here[0];
    n = n0 + last_here[1];
  }
}

Kv4AttnShape kv4_attn_shape(int sms, long long columns, long long nseq, int hk, long long keys) {
  Kv4AttnShape s;
  s.ctas = sms < kAttnMaxCtas ? sms : kAttnMaxCtas;
  s.cols = columns > 8 ? 16 : 8;
  s.warps = columns > 8 ? kAttnWarps<2> : kAttnWarps<1>;
  // CTAs that the longest batch of these bounds could use
  const long long units = nseq * hk * ((columns + s.cols - 1) / s.cols);
  const long long by_tiles = units * ((keys + kAttnKeys - 1) / kAttnKeys) / kAttnMinTiles;
  const long long most = units > by_tiles ? units : by_tiles;
  s.grid = most < 1 ? 1 : most < s.ctas ? static_cast<int>(most) : s.ctas;
  return s;
}

struct LaunchAttn {
  const Kv4AttnParams& p;
  const Kv4AttnShape& shape;
  cudaStream_t stream;
  template <int D, int GROUP, bool BF16>
  int operator()() const {
    return shape.cols == 8 ? run<D, GROUP, 1, BF16>() : run<D, GROUP, 2, BF16>();
  }
  template <int D, int GROUP, int NB, bool BF16>
  int run() const {
    using Tile = AttnTile<D, GROUP, NB>;
    constexpr int kWarps = kAttnWarps<NB>;
    const int smem = kWarps * Tile::kStages * Tile::kBytes;
    const auto kernel = kv4_attn_kernel<D, GROUP, NB, BF16>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return static_cast<int>(e);
    kernel<<<shape.grid, 32 * kWarps, smem, stream>>>(p);
    return static_cast<int>(cudaGetLastError());
  }
};
int launch_kv4_attn(const Kv4AttnParams& p, const Kv4Format& f, const Kv4AttnShape& shape,
                    cudaStream_t stream) {
  return for_kv4_format(f, LaunchAttn{p, shape, stream});
}

}  // namespace tilemix
