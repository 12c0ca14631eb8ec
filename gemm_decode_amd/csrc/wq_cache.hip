// The 8-bit key/value cache: quantise tokens as they are written, read them back.
//
// A page of a head has one power-of-two scale 2^e for its keys and one for its values: e is
// the smallest integer >= -126 with max|x| <= 127 * 2^e.  From the largest magnitude's
// fp32 form 1.m * 2^E that is E - 6 where 1.m <= 127 / 64 and E - 5 otherwise, so the
// exponent byte comes from integer operations on the bits; the codes rint(x * 2^-e) and
// the values q * 2^e are products with powers of two, without a rounding of their own.
//
//   kv_write_kernel  one workgroup per (page that is touched, head, keys or values): the new
//                    tokens' largest magnitude (16-bit integer maxima of the sign-cleared
//                    bits; a NaN or infinity wins and gives exponent byte 255), the page's
//                    exponent, then the 16-byte chunks of the page that change.  A page has
//                    one owner, so nothing is atomic and the older codes of a page whose
//                    scale grows are rewritten in place.
//   kv_read_kernel   one wave per (16-token group, head): whole 1 KB blocks in, rows out.
#include "wq_internal.h"

namespace wq {
namespace {

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

template <bool F16>
__device__ __forceinline__ float to_f32(uint32_t b) {
  return F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)b) : __uint_as_float(b << 16);
}

// exponent byte for the largest magnitude `bits` (sign-cleared, 16-bit type)
template <bool F16>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t bits) {
  if (bits >= (F16 ? 0x7C00u : 0x7F80u)) return 255u;
  const uint32_t f = __float_as_uint(to_f32<F16>(bits));
  const int E = (int)(f >> 23) - ((f & 0x7FFFFFu) <= 0x7E0000u ? 6 : 5);
  return (uint32_t)max(E, 1);
}
// 2^(127 - b) for an exponent byte b in 1 .. 253
__device__ __forceinline__ float inverse_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// codes are stored as q + 128; |x * inv| <= 127 by the choice of the exponent
__device__ __forceinline__ uint32_t code_of(float x, float inv) { return (uint32_t)((int)__builtin_rintf(x * inv) + 128); }
// four older codes of a word under a scale that grew by 2^d (shrink = 2^-d, 0 when nothing is left)
__device__ __forceinline__ uint32_t shrink_word(uint32_t w, float shrink) {
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o |= (uint32_t)((int)__builtin_rintf((float)((int)((w >> (8 * j)) & 0xFFu) - 128) * shrink) + 128) << (8 * j);
  return o;
}

struct Seq {  // rows of one sequence: first token row, count, first position
  int64_t row;
  int32_t n, start;
};
__device__ __forceinline__ Seq sequence(const KvArgs& a, int s) {
  Seq q;
  if (a.offsets) {
    const int64_t o0 = min(max((int64_t)a.offsets[s], (int64_t)0), a.tokens);
    const int64_t o1 = min(max((int64_t)a.offsets[s + 1], o0), a.tokens);
    q.row = o0;
    q.n = (int32_t)min(o1 - o0, (int64_t)a.max_tokens);
  } else {
    q.row = (int64_t)s * a.max_tokens;
    q.n = a.max_tokens;
  }
  q.start = max(a.starts[s], 0);
  // positions beyond the table (or 31 bits) are cut off
  const int64_t room = min(a.width << a.tshift, (int64_t)INT32_MAX) - q.start;
  q.n = (int32_t)max(min((int64_t)q.n, room), (int64_t)0);
  return q;
}

// grid: (pages of a sequence, heads x 2, sequences) in one dimension, heads fastest
template <bool F16, int THREADS>
__global__ __launch_bounds__(THREADS) void kv_write_kernel(KvArgs a, KvTokens kt, KvTokens vt, int span) {
  __shared__ uint32_t wave_max[THREADS / 64];
  int64_t id = blockIdx.x;
  const bool values = id & 1;
  id >>= 1;
  const int h = (int)(id % a.heads);
  id /= a.heads;
  const int pi = (int)(id % span);
  const int s = (int)(id / span);
  const Seq q = sequence(a, s);
  const int T = 1 << a.tshift;
  const int first_page = q.start >> a.tshift;
  const int64_t p0 = (int64_t)(first_page + pi) << a.tshift;      // position of the page's slot 0
  const int64_t end = (int64_t)q.start + q.n;
  if (p0 >= end) return;                                          // (also when q.n == 0)
  const int lo = (int)max((int64_t)q.start - p0, (int64_t)0);     // new slots lo .. hi - 1
  const int hi = (int)min(end - p0, (int64_t)T);
  const int page = a.table[(int64_t)s * a.width + first_page + pi];
  if ((uint32_t)page >= (uint64_t)a.pages) return;
  const KvTokens& src = values ? vt : kt;
  const int64_t row0 = q.row + (p0 + lo - q.start);               // token row of slot lo
  const uint16_t* x = src.p + row0 * src.ts + (int64_t)h * src.hs;
  const int t = threadIdx.x, D8 = a.dim / 8;

  // largest magnitude of the new tokens
  u16x2_t m = {0, 0};
  for (int i = t; i < (hi - lo) * D8; i += THREADS) {
    const uint4 w = *(const uint4*)(x + (int64_t)(i / D8) * src.ts + 8 * (i % D8));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w.x & 0x7FFF7FFFu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w.y & 0x7FFF7FFFu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w.z & 0x7FFF7FFFu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w.w & 0x7FFF7FFFu));
  }
  uint32_t mx = max((uint32_t)m.x, (uint32_t)m.y);
  uint8_t* ep = (values ? a.ve : a.ke) + (int64_t)page * a.heads + h;
  const uint32_t old_b = lo > 0 ? *ep : 0u;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d));
  if (THREADS > 64) {
    if ((t & 63) == 0) wave_max[t >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) mx = max(mx, wave_max[w]);
  }
  const uint32_t b = max(old_b, exponent_byte<F16>(mx));
  const bool grow = lo > 0 && b > old_b;
  const uint32_t d = b - old_b;
  const float shrink = !grow ? 1.f : d < 127u ? __uint_as_float((127u - d) << 23) : 0.f;
  const bool poison = b == 255u;
  const float inv = poison ? 0.f : inverse_scale(b);
  if (t == 0 && b != old_b) *ep = (uint8_t)b;

  const int DC = 4 * a.blocks;  // 16-column chunks of a token
  uint8_t* codes = (values ? a.vc : a.kc) + (((int64_t)page * a.heads + h) << a.tshift) * (16 * DC);
  if (!values) {
    // chunk = 16 columns of one token
    const int c0 = (grow ? 0 : lo) * DC;
    for (int i = c0 + t; i < hi * DC; i += THREADS) {
      const int slot = i / DC, cb = i % DC;  // columns 16 cb ..
      uint4* dst = (uint4*)(codes + (int64_t)(slot >> 4) * 256 * DC + (cb >> 2) * 1024 + (((cb & 3) << 4) | (slot & 15)) * 16);
      uint32_t o[4];
      if (slot < lo) {
        const uint4 w = *dst;
        o[0] = shrink_word(w.x, shrink);
        o[1] = shrink_word(w.y, shrink);
        o[2] = shrink_word(w.z, shrink);
        o[3] = shrink_word(w.w, shrink);
      } else {
        const uint16_t* xr = x + (int64_t)(slot - lo) * src.ts + 16 * cb;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint4 w = {0, 0, 0, 0};
          if (16 * cb + 8 * v < a.dim) w = *(const uint4*)(xr + 8 * v);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t r = 0x80808080u;
            if (!poison) {
              r = code_of(to_f32<F16>(ww[2 * e] & 0xFFFFu), inv) | code_of(to_f32<F16>(ww[2 * e] >> 16), inv) << 8 |
                  code_of(to_f32<F16>(ww[2 * e + 1] & 0xFFFFu), inv) << 16 |
                  code_of(to_f32<F16>(ww[2 * e + 1] >> 16), inv) << 24;
            }
            o[2 * v + e] = r;
          }
        }
      }
      *dst = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    // chunk = 4 columns of 4 tokens
    const int D4 = 4 * DC;
    const int c0 = ((grow ? 0 : lo) >> 2) * D4, c1 = ((hi + 3) >> 2) * D4;
    for (int i = c0 + t; i < c1; i += THREADS) {
      const int tq = i / D4, cq = i % D4;  // tokens 4 tq .., columns 4 cq ..
      uint4* dst = (uint4*)(codes + (int64_t)(tq >> 2) * 256 * DC + (cq >> 4) * 1024 + (((tq & 3) << 4) | (cq & 15)) * 16);
      uint32_t o[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
      if (4 * tq < lo) {
        const uint4 w = *dst;
        o[0] = grow ? shrink_word(w.x, shrink) : w.x;
        o[1] = grow ? shrink_word(w.y, shrink) : w.y;
        o[2] = grow ? shrink_word(w.z, shrink) : w.z;
        o[3] = grow ? shrink_word(w.w, shrink) : w.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int slot = 4 * tq + e;
        if (slot < lo || slot >= hi) continue;
        uint2 w = {0, 0};
        if (4 * cq < a.dim) w = *(const uint2*)(x + (int64_t)(slot - lo) * src.ts + 4 * cq);
        const uint32_t el[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t r = poison ? 0x80u : code_of(to_f32<F16>(el[c]), inv);
          o[c] = (o[c] & ~(0xFFu << (8 * e))) | r << (8 * e);
        }
      }
      *dst = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool F16>
__device__ __forceinline__ uint32_t value_bits(uint32_t code, float scale) {
  // the product is exact in fp32 (or overflows to an infinity, which the clamp takes back)
  const float v = (float)((int)code - 128) * scale;
  const float top = F16 ? 65504.f : __uint_as_float(0x7F7F0000u);
  const float w = v > top ? top : v < -top ? -top : v;  // (a NaN stays one)
  return F16 ? __builtin_bit_cast(uint16_t, (_Float16)w) : __builtin_bit_cast(uint16_t, (__bf16)w);
}
__device__ __forceinline__ float scale_of(uint32_t b) {
  return b == 255u ? __builtin_nanf("") : __uint_as_float(b << 23);
}

// one wave per (16-token group, head): grid-linear waves, heads fastest
template <bool F16>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a, KvTokens kt, KvTokens vt, int span, int64_t waves) {
  int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= waves) return;
  const int lane = threadIdx.x & 63;
  const int h = (int)(id % a.heads);
  id /= a.heads;
  const int gi = (int)(id % span);
  const int s = (int)(id / span);
  const Seq q = sequence(a, s);
  const int64_t g0 = ((int64_t)(q.start >> 4) + gi) << 4;  // position of the group's first token
  const int64_t end = (int64_t)q.start + q.n;
  if (g0 >= end) return;
  const int page = a.table[(int64_t)s * a.width + (g0 >> a.tshift)];
  const bool in_pool = (uint32_t)page < (uint64_t)a.pages;
  const int64_t ph = (int64_t)(in_pool ? page : 0) * a.heads + h;
  const float ks = in_pool ? scale_of(a.ke[ph]) : scale_of(255u), vs = in_pool ? scale_of(a.ve[ph]) : scale_of(255u);
  const int64_t off = ((ph << a.tshift) + (g0 & ((1 << a.tshift) - 1))) * (64 * a.blocks) + lane * 16;
  for (int blk = 0; blk < a.blocks; ++blk) {
    const uint4 kw = *(const uint4*)(a.kc + off + blk * 1024), vw = *(const uint4*)(a.vc + off + blk * 1024);
    {  // keys: 16 columns of token lane % 16
      const int64_t pos = g0 + (lane & 15);
      const int d = 64 * blk + 16 * (lane >> 4);
      if (pos >= q.start && pos < end) {
        uint16_t* y = kt.p + (q.row + (pos - q.start)) * kt.ts + (int64_t)h * kt.hs + d;
        const uint32_t ww[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (d + 8 * v < a.dim) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t w = ww[2 * v + (j >> 1)] >> (16 * (j & 1));
              o[j] = value_bits<F16>(w & 0xFFu, ks) | value_bits<F16>((w >> 8) & 0xFFu, ks) << 16;
            }
            *(uint4*)(y + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
          }
      }
    }
    {  // values: 4 columns of the tokens 4 (lane / 16) ..
      const int d = 64 * blk + 4 * (lane & 15);
      const uint32_t ww[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t pos = g0 + 4 * (lane >> 4) + e;
        if (pos >= q.start && pos < end && d < a.dim) {
          uint16_t* y = vt.p + (q.row + (pos - q.start)) * vt.ts + (int64_t)h * vt.hs + d;
          uint32_t o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            o[j] = value_bits<F16>((ww[2 * j] >> (8 * e)) & 0xFFu, vs) |
                   value_bits<F16>((ww[2 * j + 1] >> (8 * e)) & 0xFFu, vs) << 16;
          *(uint2*)y = make_uint2(o[0], o[1]);
        }
      }
    }
  }
}

// units of `unit` tokens that a sequence's rows touch at most, whatever its first position
int64_t touched(int64_t tokens, int unit) { return (tokens + 2 * unit - 2) / unit; }

}  // namespace

wq_status launch_kv_write(const KvArgs& a, const KvTokens& k, const KvTokens& v, bool f16, hipStream_t s) {
  const int64_t span = touched(a.max_tokens, 1 << a.tshift);
  const __int128 blocks = (__int128)a.seqs * span * a.heads * 2;
  if (blocks > INT32_MAX) return fail(WQ_ERR_UNSUPPORTED, "wq_kv_write: too many pages for one call");
  auto go = [&](auto kernel, int threads) { kernel<<<(unsigned)blocks, threads, 0, s>>>(a, k, v, (int)span); };
  if ((int64_t)a.max_tokens * a.dim <= 2048) f16 ? go(kv_write_kernel<true, 64>, 64) : go(kv_write_kernel<false, 64>, 64);
  else f16 ? go(kv_write_kernel<true, 256>, 256) : go(kv_write_kernel<false, 256>, 256);
  WQ_HIP_CHECK(hipGetLastError());
  return WQ_OK;
}

wq_status launch_kv_read(const KvArgs& a, const KvTokens& k, const KvTokens& v, bool f16, hipStream_t s) {
  const int64_t span = touched(a.max_tokens, 16);
  const __int128 waves = (__int128)a.seqs * span * a.heads;
  if (span > INT32_MAX || (waves + 3) / 4 > INT32_MAX) return fail(WQ_ERR_UNSUPPORTED, "wq_kv_read: too many tokens for one call");
  const unsigned blocks = (unsigned)((waves + 3) / 4);
  if (f16) kv_read_kernel<true><<<blocks, 256, 0, s>>>(a, k, v, (int)span, (int64_t)waves);
  else kv_read_kernel<false><<<blocks, 256, 0, s>>>(a, k, v, (int)span, (int64_t)waves);
  WQ_HIP_CHECK(hipGetLastError());
  return WQ_OK;
}

}  // namespace wq
