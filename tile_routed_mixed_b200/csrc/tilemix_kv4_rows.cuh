// Rows into and out of the paged 4-bit cache (tilemix_kv4_append,
// tilemix_kv4_gather).
//
// Both are one pass over memory, a thread to a chunk of 8 channels: 16 bytes of
// activations against one 4-byte word of codes.  A group of channels
// is 4, 8 or 16 neighbouring lanes, which take its largest magnitude with
// shuffles; nothing is staged.
//
// Rounding.  s = a / 7 is never within 2^-15 (relative) of a midpoint of the
// scale's type, as 7 divides no midpoint of an 11-bit significand, so one fp32
// multiply by 1/7 and one conversion give the correctly rounded s.  The
// quotient x / s of two significands of at most 11 bits is a half-integer or
// at least 1 / 4094 away from every half-integer below 7.  The reciprocal
// product is within 2^-19 of the quotient, so rounding it to a multiple of
// 2^-12 moves no quotient across a half-integer and puts every tie exactly
// on one, and the second rounding (to an integer, ties to even) gives
// rne(x / s) as IEEE division would.
//
// Measured (B200): 32768 tokens of 8 heads of 128 in, 172 MB in 36 us; out
// again 37 us; 12 ragged sequences of up to 16384 tokens of 4 heads out, 243 MB
// in 49 us: 4.7 to 4.9 TB/s, 0.72 to 0.75 of the measured copy rate.  Issue bounds
// them: 0.78 of the slots (ALU 0.67 in, 0.77 out), DRAM below a half.  Before (48
// and 45 us) a chunk found its token, head and place by itself: so a thread
// keeps one place of a row over its tokens, quotients outside +-7 and subnormal
// scales have a path of their own, and a product of code and scale is one packed
// multiplication in the type, rounded once.
// Included by tilemix_kv4.cu.
#pragma once

namespace tilemix {

constexpr int kRowThreads = 256;
// Chunks from which a thread takes four tokens, loaded together: two full waves
// of one each.  Above, one / four: 32768 tokens in 49 / 36 us, out 58 / 37, the
// ragged batch out 78 / 49.  Below, one each spreads the rows over more SMs: 8
// tokens in 1.3 / 1.8 us, one sequence of 1000 out 1.9 / 2.3.
constexpr long long kRowsWide = 148LL * 2048 * 2;

namespace kv4 {

// The codes of nibbles in both halves of a word, as fp16 pairs.
__device__ __forceinline__ uint32_t or_1024(uint32_t x, uint32_t mask) {  // (x & mask) | 0x64006400
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(y) : "r"(x), "r"(mask));
  return y;
}
__device__ __forceinline__ uint32_t code_low(uint32_t x) {  // bits 0 .. 3: 1024 + u - 1032
  uint32_t y = or_1024(x, 0x000F000Fu);
  asm("add.f16x2 %0, %0, %1;" : "+r"(y) : "r"(0xE408E408u));
  return y;
}
__device__ __forceinline__ uint32_t code_high(uint32_t x) {  // bits 4 .. 7: (1024 + 16 u) / 16 - 72
  uint32_t y = or_1024(x, 0x00F000F0u);
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(y) : "r"(0x2C002C00u), "r"(0xD480D480u));
  return y;
}

// Two packed values of the activations' type to fp32.
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool BF16>
__device__ __forceinline__ float unpack1(uint32_t bits) {
  if constexpr (BF16)
    return __uint_as_float(bits << 16);
  else
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack1(float x) {
  if constexpr (BF16)
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else
    return __half_as_ushort(__float2half_rn(x));
}
// 1 / x to within an ulp (x normal).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bit pattern of the type's infinity: magnitudes from it on are not finite.
template <bool BF16>
constexpr uint32_t kInfBits = BF16 ? 0x7f80u : 0x7c00u;

// Largest magnitude of a chunk, as a bit pattern (magnitudes of a type are
// ordered like their patterns, NaNs above all).
__device__ __forceinline__ uint32_t absmax_bits(const uint4& u) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
  return max(a & 0xffffu, a >> 16);
}

// The eight codes + 8 of a chunk as nibbles, channel 0 lowest.  r = 4096 / s (0
// for s = 0).  RARE: s is subnormal (or zero); quotients may then lie beyond
// +-7, and up is the power of two that r's s was multiplied by.
constexpr float kShift = 12582912.0f;  // 1.5 * 2^23: x + kShift is rne(x) + kShift
template <bool BF16, bool RARE>
__device__ __forceinline__ uint32_t code_word(const uint4& u, float r, float up) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<BF16>(w[i]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float c = (j ? x.y : x.x) * (RARE ? up : 1.0f);
      // 4096 x / s, rounded to an integer
      float t = __fadd_rn(__fmaf_rn(c, r, kShift), -kShift);
      if (RARE) t = fminf(fmaxf(t, -28672.0f), 28672.0f);
      // its 2^-12th, rounded to an integer, + 8: the low byte of the sum
      b[2 * i + j] = __float_as_uint(__fmaf_rn(t, 0x1p-12f, kShift + 8.0f));
    }
  }
  const uint32_t even = __byte_perm(__byte_perm(b[0], b[2], 0x0040), __byte_perm(b[4], b[6], 0x0040), 0x5410);
  const uint32_t odd = __byte_perm(__byte_perm(b[1], b[3], 0x0040), __byte_perm(b[5], b[7], 0x0040), 0x5410);
  return even + (odd << 4);
}

// The eight values of a word of codes, scaled: the product of a code and a
// scale in the type itself is rounded once.
template <bool BF16>
__device__ __forceinline__ uint4 values_of(uint32_t w, uint32_t scale) {
  const uint32_t s2 = scale | (scale << 16);
  uint32_t p[4];  // channels i and i + 4
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // 128 + u, less 136
      uint32_t c = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
      asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(c) : "r"(0xC308C308u));
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(c), "r"(s2));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (i & 1) ? code_high(w >> (8 * (i / 2))) : code_low(w >> (8 * (i / 2)));
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(c), "r"(s2));
    }
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// Place of a row's 32-bit word of K holding channels 8w .. 8w + 7.
template <int D>
__device__ __forceinline__ int k_place(int w) {
  return (w & 3) * (D / 32) + (w >> 2);
}

}  // namespace kv4

// A thread has one place of one head's rows (blockIdx.y: head; blockIdx.z: K or
// V) and U tokens, so that what follows from the place is found once; the U
// tokens' chunks are all loaded before the first is coded.
template <int D, int GROUP, bool BF16, int U>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendParams p) {
  constexpr int kChunks = D / 8;  // of a row: 8 or 16, so a warp holds whole rows
  constexpr int T = D / 32, kTokens = kRowThreads / kChunks;  // tokens of a sweep
  const bool is_v = blockIdx.z != 0;
  const int w = threadIdx.x % kChunks, head = blockIdx.y;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const int token0 = blockIdx.x * (U * kTokens) + threadIdx.x / kChunks;
  const uint8_t* src = (is_v ? p.v : p.k) + (head * kChunks + w) * 16;
  uint4 data[U];
  int slots[U];
#pragma unroll
  for (int x = 0; x < U; ++x) {
    const int token = token0 + x * kTokens;
    const bool live = token < p.n;
    data[x] = make_uint4(0u, 0u, 0u, 0u);
    slots[x] = -1;
    if (live) {
      data[x] = __ldg(reinterpret_cast<const uint4*>(src + token * stride));
      slots[x] = __ldg(p.slots + token);
    }
  }
  // V's halfwords 2w and 2w + 1 lie apart: halfword 8t + g at place g T + t.  The
  // lane four on holds the same places of the next t: each of the two lanes sends
  // one half and keeps a whole 32-bit word.
  const int t = w >> 2;
  const int place = is_v ? (2 * (w & 3) + (t & 1)) * (T / 2) + (t >> 1) : kv4::k_place<D>(w);
  uint8_t* const codes = (is_v ? p.pool.v_codes : p.pool.k_codes) + place * 4;
  uint8_t* const scales = (is_v ? p.pool.v_scale : p.pool.k_scale) + 2 * (w / (GROUP / 8));
  const int sh = p.pool.page_shift, in_page = (1 << sh) - 1;
#pragma unroll
  for (int x = 0; x < U; ++x) {
    const uint4 u = data[x];
    uint32_t a = kv4::absmax_bits(u);
#pragma unroll
    for (int by = GROUP / 16; by > 0; by >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, by));
    const bool finite = a < kv4::kInfBits<BF16>;
    const uint32_t sbits = finite ? kv4::pack1<BF16>(kv4::unpack1<BF16>(a) * (1.0f / 7.0f))
                                  : kv4::kInfBits<BF16> + 1u;
    uint32_t word = 0x88888888u;
    if (finite && sbits >= (BF16 ? 0x0e00u : 0x0400u)) {  // s >= 2^-99 (2^-14): normal
      word = kv4::code_word<BF16, false>(u, kv4::rcp(kv4::unpack1<BF16>(sbits)) * 4096.0f, 1.0f);
    } else if (finite && sbits != 0) {
      const float up = BF16 ? 0x1p64f : 1.0f;  // so that 4096 / s stays finite
      word = kv4::code_word<BF16, true>(u, kv4::rcp(kv4::unpack1<BF16>(sbits) * up) * 4096.0f, up);
    }
    if (is_v) {
      const uint32_t other =
          __shfl_xor_sync(0xffffffffu, (t & 1) ? word & 0xffffu : word >> 16, 4);
      word = (t & 1) ? __byte_perm(other, word, 0x7610) : __byte_perm(word, other, 0x5410);
    }
    const int slot = slots[x], page = slot >> sh;  // -1 for -1
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pool.num_pages)) {
      const int64_t row = ((static_cast<int64_t>(page) * p.pool.hk + head) << sh) + (slot & in_page);
      *reinterpret_cast<uint32_t*>(codes + row * (D / 2)) = word;
      if (w % (GROUP / 8) == 0)
        *reinterpret_cast<unsigned short*>(scales + row * (2 * (D / GROUP))) =
            static_cast<unsigned short>(sbits);
    } else if (slot != -1) {
      atomicOr(&g_kv4_status, kStatusBadPages);
    }
  }
}

// blockIdx.y: sequence; blockIdx.z: head, K before V; the CTAs of blockIdx.x stride
// over the sequence's tokens.  A thread takes the 32-bit word at its own place of
// a row (of V, half of two words: it exchanges one with the lane that has their
// other halves), U tokens' words before it writes the first.
template <int D, int GROUP, bool BF16, int U>
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const Kv4GatherParams p) {
  constexpr int kChunks = D / 8;
  constexpr int T = D / 32, kTokens = kRowThreads / kChunks;
  const int hk = p.pool.hk, sh = p.pool.page_shift, in_page = (1 << sh) - 1;
  const bool is_v = static_cast<int>(blockIdx.z) >= hk;
  const int head = is_v ? blockIdx.z - hk : blockIdx.z, s = blockIdx.y;
  const long long top = min(static_cast<long long>(p.max_pages) << sh, 0x7f000000LL);
  const int have = __ldg(p.seq_len + s);
  const int len = static_cast<int>(min(static_cast<long long>(max(have, 0)), top));
  const long long out0 = __ldg(p.out_start + s);
  // positions whose rows lie inside the output
  const int from = static_cast<int>(max(0LL, min(-out0, static_cast<long long>(len))));
  const int to = static_cast<int>(max(0LL, min(p.rows - out0, static_cast<long long>(len))));
  bool bad = have != len || from > 0 || to < len;
  const int at = threadIdx.x % kChunks;
  // K: place q T + t holds word 4t + q; V: place g (T / 2) + t / 2 makes, with the
  // lane of g ^ 1, words 4t + g / 2 of both t, of which it keeps t + (g & 1)
  const bool odd = (at / (T / 2)) & 1;
  const int w = is_v ? 4 * (2 * (at % (T / 2)) + odd) + at / T : 4 * (at % T) + at / T;
  const uint8_t* const codes = (is_v ? p.pool.v_codes : p.pool.k_codes) + at * 4;
  const uint8_t* const scales = (is_v ? p.pool.v_scale : p.pool.k_scale) + 2 * (w / (GROUP / 8));
  uint8_t* const out = (is_v ? p.v : p.k) + (head * kChunks + w) * 16;
  const int64_t out_row = static_cast<int64_t>(hk) * (2 * D);
  const int32_t* const table = p.block_table + static_cast<size_t>(s) * p.max_pages;
  const int step = gridDim.x * (U * kTokens);
  for (int base = blockIdx.x * (U * kTokens); base < len; base += step) {
    const int pos0 = base + threadIdx.x / kChunks;
    uint32_t word[U], scale[U];
    int page[U];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int pos = pos0 + x * kTokens;
      page[x] = pos >= from && pos < to ? __ldg(table + (pos >> sh)) : -1;
      if (pos >= from && pos < to) bad |= page[x] < 0 || page[x] >= p.pool.num_pages;
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      word[x] = scale[x] = 0u;
      if (static_cast<unsigned>(page[x]) < static_cast<unsigned>(p.pool.num_pages)) {
        const int64_t row = ((static_cast<int64_t>(page[x]) * hk + head) << sh) +
                            ((pos0 + x * kTokens) & in_page);
        word[x] = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (D / 2)));
        scale[x] = __ldg(reinterpret_cast<const unsigned short*>(scales + row * (2 * (D / GROUP))));
      } else {
        page[x] = -1;
      }
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      uint32_t v = word[x];
      if (is_v) {
        // lanes of one row: an even g sends its high half, an odd one its low
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? v & 0xffffu : v >> 16, T / 2);
        v = odd ? __byte_perm(other, v, 0x7610) : __byte_perm(v, other, 0x5410);
      }
      if (page[x] >= 0)
        *reinterpret_cast<uint4*>(out + (out0 + pos0 + x * kTokens) * out_row) =
            kv4::values_of<BF16>(v, scale[x]);
    }
  }
  if (bad) atomicOr(&g_kv4_status, kStatusBadPages);
}

// Calls fn.template operator()<D, GROUP, BF16>() for the format.
template <class Fn>
int for_kv4_format(const Kv4Format& f, Fn fn) {
  if (f.d == 128) {
    if (f.group == 32) return f.bf16 ? fn.template operator()<128, 32, true>() : fn.template operator()<128, 32, false>();
    if (f.group == 64) return f.bf16 ? fn.template operator()<128, 64, true>() : fn.template operator()<128, 64, false>();
    if (f.group == 128) return f.bf16 ? fn.template operator()<128, 128, true>() : fn.template operator()<128, 128, false>();
  } else if (f.d == 64) {
    if (f.group == 32) return f.bf16 ? fn.template operator()<64, 32, true>() : fn.template operator()<64, 32, false>();
    if (f.group == 64) return f.bf16 ? fn.template operator()<64, 64, true>() : fn.template operator()<64, 64, false>();
  }
  return cudaErrorInvalidValue;
}

struct LaunchAppend {
  const Kv4AppendParams& p;
  cudaStream_t stream;
  template <int D, int GROUP, bool BF16>
  int operator()() const {
    const long long chunks = static_cast<long long>(p.n) * p.pool.hk * (D / 8);
    return chunks < kRowsWide ? run<D, GROUP, BF16, 1>() : run<D, GROUP, BF16, 4>();
  }
  template <int D, int GROUP, bool BF16, int U>
  int run() const {
    constexpr int kTokens = U * kRowThreads / (D / 8);
    const dim3 grid((p.n + kTokens - 1) / kTokens, p.pool.hk, 2);
    kv4_append_kernel<D, GROUP, BF16, U><<<grid, kRowThreads, 0, stream>>>(p);
    return static_cast<int>(cudaGetLastError());
  }
};
int launch_kv4_append(const Kv4AppendParams& p, const Kv4Format& f, cudaStream_t stream) {
  return for_kv4_format(f, LaunchAppend{p, stream});
}

struct LaunchGather {
  const Kv4GatherParams& p;
  cudaStream_t stream;
  template <int D, int GROUP, bool BF16>
  int operator()() const {
    const long long chunks = static_cast<long long>(p.rows) * p.pool.hk * (D / 8);
    return chunks < kRowsWide ? run<D, GROUP, BF16, 1>() : run<D, GROUP, BF16, 4>();
  }
  template <int D, int GROUP, bool BF16, int U>
  int run() const {
    // one sweep of a sequence of the average length
    constexpr int kTokens = U * kRowThreads / (D / 8);
    int sweep = (p.rows / p.nseq + kTokens - 1) / kTokens;
    sweep = sweep < 1 ? 1 : sweep > 16384 ? 16384 : sweep;
    const dim3 grid(sweep, p.nseq, 2 * p.pool.hk);
    kv4_gather_kernel<D, GROUP, BF16, U><<<grid, kRowThreads, 0, stream>>>(p);
    return static_cast<int>(cudaGetLastError());
  }
};
int launch_kv4_gather(const Kv4GatherParams& p, const Kv4Format& f, cudaStream_t stream) {
  return for_kv4_format(f, LaunchGather{p, stream});
}

}  // namespace tilemix
