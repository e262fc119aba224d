// Key/value cache held in 4 bits: quantising rows as they are written, reading them back, and
// attention over the cache.
//
// A page holds 2^page_shift positions of one sequence; for each kv head in turn
//   K codes  [page][D / 2]          byte i of a position: d = 2 i low nibble, 2 i + 1 high
//   K scales [page][D / G] bf16
//   V codes  [page / 8][D][4]       byte i of (block, d): position 2 i of the block low, 2 i + 1 high
//   V scales [page / 8][D / G][8] bf16
// Each operand is packed along the axis its product sums over, as the packed weights are: scores
// sum over d, outputs over positions.  A lane's operand of a 16x16x32 matrix instruction is 8
// values along that axis, so one dword of codes decodes in place to one operand and no value
// changes lanes.
#include <float.h>
#include <math.h>

#include "dqg_device.hpp"
#include "dqg_internal.hpp"

namespace dqg {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr int ST_PAGE = 1;    // status bit 0: a page id outside [0, num_pages)
constexpr int ST_LENGTH = 2;  // status bit 1: a length beyond the table's positions

__device__ __forceinline__ void report(int* status, int bit) {
  if (status) atomicOr(status, bit);
}

// The last i of 0 .. n - 1 with key(i) <= x, where key ascends from key(0) <= x: 64 candidates a
// step.  Uniform over the wavefront; in range for any keys.
template <class F>
__device__ __forceinline__ int last_at_most(int n, int x, F key) {
  const int lane = threadIdx.x & 63;
  int lo = 0, end = n;
  while (end - lo > 1) {
    const int step = (end - lo + 63) >> 6, i = lo + lane * step;
    const int c = __popcll(__ballot(i < end && key(i) <= x));
    lo += max(c - 1, 0) * step;
    end = min(lo + step, end);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
// The sequence that slot `slot` falls to when sequence b's slots start at first(cu[b]) + b * per.
template <class F>
__device__ __forceinline__ int seq_of_slot(const Kv4Where& w, int slot, int per, F first) {
  return last_at_most(w.B, slot,
                      [&](int b) { return first(min(max(w.cu[b], 0), w.T)) + b * per; });
}

struct Seq {
  int row0, n;   // rows row0 .. row0 + n - 1
  int len, cap;  // positions, and how many of them the table has room for
};
__device__ __forceinline__ Seq seq_at(const Kv4Where& w, int b) {
  Seq s;
  s.row0 = min(max(w.cu[b], 0), w.T);
  s.n = min(max(w.cu[b + 1], s.row0), w.T) - s.row0;
  s.len = min(max(w.lens[b], 0), 0x7FFF0000);
  s.cap = w.max_pages << w.page_shift;
  return s;
}

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}

// the value of another lane: of lane ^ 1, of lane ^ 2, of the mirror image within 8 lanes, within 16
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_MIRROR8 = 0x141, DPP_MIRROR16 = 0x140;
template <int C>
__device__ __forceinline__ uint32_t dpp_of(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, C, 0xF, 0xF, true);
}

// ---- quantisation -----------------------------------------------------------------------
// s = bf16(amax / c), code = nearest(x / s).  x and s have 8 significant bits, so a quotient that
// is no tie is at least 1 / 1020 away from every tie of either grid; fma(x, 1 / s, 1536) rounds
// the quotient to multiples of 2^-13 with an error (reciprocal and fma, below 2^-18) that
// cannot carry it across one, and lands exactly on a tie where the true quotient is one.  The
// codes are therefore those of an exact division.
struct GroupScale {
  uint16_t bits;  // bf16 scale
  float inv;      // 1 / scale, or 0
};
template <int FMT>
__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits) {
  GroupScale g;
  const float a = __uint_as_float(amax_bits << 16);
  // (a / c is at least 1 / 3584 of itself away from a rounding tie: the product rounds alike)
  const uint32_t bits = f32_to_bf16(a * (FMT == FMT_INT4 ? 1.0f / 7.0f : 1.0f / 6.0f));
  const float inv = __builtin_amdgcn_rcpf(__uint_as_float(bits << 16));
  const bool small = amax_bits < 0x0D80u;  // below 2^-100
  const bool bad = amax_bits >= 0x7F80u;   // a NaN or an infinity: the group reads back as NaN
  g.bits = (uint16_t)(bad ? 0x7FC0u : small ? 0u : bits);
  g.inv = bad || small ? 0.0f : inv;
  return g;
}
// the code of x in the low 4 bits (INT4; the others hold rubbish)
__device__ __forceinline__ uint32_t int4_code(float x, float inv) {
  // 12582912 = 1.5 * 2^23: the sum's low bits are the rounded quotient (ties to even) + 8
  return __float_as_uint(fmaf(x, inv, 1536.0f) + (12582912.0f + 8.0f - 1536.0f));
}
// (with the sign of x where it is zero: FP4 codes keep the sign)
__device__ __forceinline__ float snapped(float x, float inv) {
  return copysignf(fmaf(x, inv, 1536.0f) - 1536.0f, x);
}
// codes of 8 values, first in the low nibble
template <int FMT>
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], const float (&inv)[8]) {
  uint32_t w = 0;
  if constexpr (FMT == FMT_INT4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (int4_code(x[i], inv[i]) & 15u) << (4 * i);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, snapped(x[0], inv[0]), snapped(x[1], inv[1]), 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, snapped(x[2], inv[2]), snapped(x[3], inv[3]), 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, snapped(x[4], inv[4]), snapped(x[5], inv[5]), 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, snapped(x[6], inv[6]), snapped(x[7], inv[7]), 1.0f, 3);
  }
  return w;
}
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, float (&x)[8]) {
  if constexpr (FMT == FMT_INT4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __uint_as_float(((w >> (4 * i)) & 15u) | 0x4B000000u) - 8388616.0f;
  } else {
    const f32x2_t a = fp4_pair_f32<0>(w), b = fp4_pair_f32<1>(w);
    const f32x2_t c = fp4_pair_f32<2>(w), d = fp4_pair_f32<3>(w);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
  }
}

// Rows of one block of 8 aligned positions that the call writes or reads.  Rows before position
// 0 (idle slots of a padded batch hold no position) lie in blocks of negative positions.
struct Block {
  int head, slot;  // slot: first position of the block within its page
  int lo, hi;      // the call's rows are positions lo .. hi - 1 of the block
  int64_t row;     // row of the block's first position (may be before the sequence's rows)
  uint8_t* base;   // the head's part of the page
  bool held;       // the block has a place in the cache
};
// Slots of a sequence: n rows touch at most floor((n + 14) / 8) blocks, and
// floor(cu[b + 1] / 8) - floor(cu[b] / 8) + 2 >= ceil((n + 9) / 8) is at least that.
__device__ __forceinline__ bool block_at(const Kv4Where& w, int slot, int head, Block& o) {
  const int b = seq_of_slot(w, slot, 2, [](int c) { return c >> 3; });
  const Seq s = seq_at(w, b);
  const int first = s.len - s.n;  // position of row 0
  const int pos0 = (first & ~7) + 8 * (slot - ((s.row0 >> 3) + 2 * b));
  if (s.n <= 0 || pos0 >= s.len || pos0 + 8 <= first) return false;
  o.head = head;
  o.lo = max(first - pos0, 0);
  o.hi = min(s.len - pos0, 8);
  o.row = (int64_t)s.row0 + (pos0 - first);
  o.slot = pos0 & ((1 << w.page_shift) - 1);
  o.base = w.cache;
  o.held = false;
  if (pos0 < 0) return true;
  int bad = ST_LENGTH;
  if (pos0 < s.cap) {
    const int page = w.table[(int64_t)b * w.max_pages + (pos0 >> w.page_shift)];
    bad = ST_PAGE;
    if (page >= 0 && page < w.num_pages) {
      o.base += page * w.page_bytes + (int64_t)head * w.head_bytes;
      o.held = true;
    }
  }
  if (!o.held && (threadIdx.x & 63) == 0) report(w.status, bad);
  return true;
}

// Byte offsets inside a head's part of a page.
template <int D>
struct Layout {
  int n_shift;  // log2(D / G)
  int ks, vc, vs;
  __device__ __forceinline__ Layout(const Kv4Where& w) {
    constexpr int lg = D == 64 ? 6 : D == 128 ? 7 : 8;
    n_shift = lg - w.group_shift;
    const int codes = (D / 2) << w.page_shift, scales = 2 << (w.page_shift + n_shift);
    ks = codes;
    vc = codes + scales;
    vs = 2 * codes + scales;
  }
};

// ---- write --------------------------------------------------------------------------------
// K: 16 values of one position a lane (32-byte loads, 8-byte stores).  V: 2 columns of all 8
// positions a lane, so that the lane owns whole dwords of codes; a block that the call does not
// fill keeps the other positions' nibbles.  A wavefront takes K or V of one block and head: the
// most wavefronts, for a single row as for a prompt.
// Instructions bound it, not memory (per wavefront about 250 for K, 450 for V and 2 KB of rows):
// maxima cross lanes by DPP, loads and scales are free of branches.  12171 rows of 4 heads of 128 in
// 3 prompts: 10.2 us (32 MB: 3.1 TB/s, of the 5.1 of a large copy; with branches and LDS exchanges
// 13.2); one row: 3.5 us.
template <int D, int FMT>
__global__ __launch_bounds__(256) void kv4_write_kernel(Kv4RowsArgs a, int n_units) {
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= n_units) return;
  const int lane = threadIdx.x & 63;
  const bool is_v = unit & 1;
  const int hs = unit >> 1;
  Block o;
  if (!block_at(a.w, hs / a.w.Hkv, hs % a.w.Hkv, o) || !o.held) return;
  const Layout<D> L(a.w);
  const int gs = a.w.group_shift;
  if (!is_v) {
    constexpr int LT = D / 16;  // lanes a position
#pragma unroll
    for (int it = 0; it < (8 * LT + 63) / 64; ++it) {
      const int item = it * 64 + lane, t = item / LT, d0 = (item % LT) * 16;
      const bool on = t >= o.lo && t < o.hi;
      uint4 x[2] = {};
      if (on) {
        const uint4* p = reinterpret_cast<const uint4*>(a.k + (o.row + t) * a.k_stride +
                                                        (int64_t)o.head * D + d0);
        x[0] = p[0];
        x[1] = p[1];
      }
      const uint32_t u[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = pk_max_u16(m, u[i] & 0x7FFF7FFFu);
      uint32_t am = max(m & 0xFFFFu, m >> 16);
      am = max(am, dpp_of<DPP_XOR1>(am));
      if (gs == 7) {
        am = max(am, dpp_of<DPP_XOR2>(am));
        am = max(am, dpp_of<DPP_MIRROR8>(am));
      }
      const GroupScale g = group_scale<FMT>(am);
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8], inv[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_lo(u[4 * h + i]);
          f[2 * i + 1] = bf16_hi(u[4 * h + i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) inv[i] = g.inv;
        c[h] = encode8<FMT>(f, inv);
      }
      if (on) {
        *reinterpret_cast<uint2*>(o.base + (o.slot + t) * (D / 2) + d0 / 2) = make_uint2(c[0], c[1]);
        if ((d0 & ((1 << gs) - 1)) == 0)
          *reinterpret_cast<uint16_t*>(o.base + L.ks +
                                       2 * (((o.slot + t) << L.n_shift) + (d0 >> gs))) = g.bits;
      }
    }
  } else {
#pragma unroll
    for (int it = 0; it < (D + 127) / 128; ++it) {
      const bool mine = it * 128 + 2 * lane < D;
      const int d0 = mine ? it * 128 + 2 * lane : 0;
      uint32_t u[8];
      const uint16_t* row = a.v + (o.row + o.lo) * a.v_stride + (int64_t)o.head * D;
#pragma unroll
      for (int t = 0; t < 8; ++t) {  // (a position that is not the call's: the nearest that is)
        if (t > 0) row += t > o.lo && t < o.hi ? a.v_stride : 0;
        u[t] = *reinterpret_cast<const uint32_t*>(row + (uint32_t)d0);
      }
      const bool whole = o.lo == 0 && o.hi == 8;
      float inv[8];
      uint16_t bits[8];
#pragma unroll
      for (int t = 0; t < 8; t += 2) {  // two positions' maxima in one dword
        const uint32_t x = u[t] & 0x7FFF7FFFu, y = u[t + 1] & 0x7FFF7FFFu;
        uint32_t m = max(x & 0xFFFFu, x >> 16) | (max(y & 0xFFFFu, y >> 16) << 16);
        m = pk_max_u16(m, dpp_of<DPP_XOR1>(m));
        m = pk_max_u16(m, dpp_of<DPP_XOR2>(m));
        m = pk_max_u16(m, dpp_of<DPP_MIRROR8>(m));
        m = pk_max_u16(m, dpp_of<DPP_MIRROR16>(m));
        if (gs == 7) {
          m = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, 16));
          m = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, 32));
        }
        const GroupScale g0 = group_scale<FMT>(m & 0xFFFFu), g1 = group_scale<FMT>(m >> 16);
        inv[t] = g0.inv; bits[t] = g0.bits;
        inv[t + 1] = g1.inv; bits[t + 1] = g1.bits;
      }
      float f0[8], f1[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        f0[t] = bf16_lo(u[t]);
        f1[t] = bf16_hi(u[t]);
      }
      uint2 c = make_uint2(encode8<FMT>(f0, inv), encode8<FMT>(f1, inv));
      if (mine) {
        uint2* p = reinterpret_cast<uint2*>(o.base + L.vc + ((o.slot >> 3) * D + d0) * 4);
        if (!whole) {
          const uint32_t keep = ~(uint32_t)((((uint64_t)1 << (4 * o.hi)) - 1) &
                                            ~(((uint64_t)1 << (4 * o.lo)) - 1));
          const uint2 old = *p;
          c.x = (c.x & ~keep) | (old.x & keep);
          c.y = (c.y & ~keep) | (old.y & keep);
        }
        *p = c;
        if ((d0 & ((1 << gs) - 1)) == 0) {
          uint16_t* s = reinterpret_cast<uint16_t*>(
              o.base + L.vs + 16 * (((o.slot >> 3) << L.n_shift) + (d0 >> gs)));
          if (whole) {
            uint4 w;
            w.x = bits[0] | (uint32_t)bits[1] << 16;
            w.y = bits[2] | (uint32_t)bits[3] << 16;
            w.z = bits[4] | (uint32_t)bits[5] << 16;
            w.w = bits[6] | (uint32_t)bits[7] << 16;
            *reinterpret_cast<uint4*>(s) = w;
          } else {
#pragma unroll
            for (int t = 0; t < 8; ++t)
              if (t >= o.lo && t < o.hi) s[t] = bits[t];
          }
        }
      }
    }
  }
}

// ---- read ---------------------------------------------------------------------------------
// The same lanes the other way round.  Rows without a place in the cache (before position 0, or
// behind the table, or in a page that is not there) read as zeros.  Bound by memory: 32768 rows of
// 4 heads of 128 16.7 us (86 MB: 5.1 TB/s, as a large copy); the 12171 rows above 9.3 us.
template <int D, int FMT>
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4RowsArgs a, int n_units) {
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= n_units) return;
  const int lane = threadIdx.x & 63;
  const bool is_v = unit & 1;
  const int hs = unit >> 1;
  Block o;
  if (!block_at(a.w, hs / a.w.Hkv, hs % a.w.Hkv, o)) return;
  const Layout<D> L(a.w);
  const int gs = a.w.group_shift;
  constexpr uint32_t zeros = FMT == FMT_INT4 ? 0x88888888u : 0u;  // codes of 0
  if (!is_v) {
    constexpr int LT = D / 16;
#pragma unroll
    for (int it = 0; it < (8 * LT + 63) / 64; ++it) {
      const int item = it * 64 + lane, t = item / LT, d0 = (item % LT) * 16;
      if (t < o.lo || t >= o.hi) continue;
      uint2 c = make_uint2(zeros, zeros);
      float s = 0.0f;
      if (o.held) {
        c = *reinterpret_cast<const uint2*>(o.base + (o.slot + t) * (D / 2) + d0 / 2);
        s = bf16_to_f32(*reinterpret_cast<const uint16_t*>(
            o.base + L.ks + 2 * (((o.slot + t) << L.n_shift) + (d0 >> gs))));
      }
      float f[16];
      {
        float x[8], y[8];
        decode8<FMT>(c.x, x);
        decode8<FMT>(c.y, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = x[i] * s;
          f[8 + i] = y[i] * s;
        }
      }
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bf16x2_t h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
        r[i] = __builtin_bit_cast(uint32_t, h);
      }
      uint4* p = reinterpret_cast<uint4*>(a.k_out + (o.row + t) * a.k_stride +
                                          (int64_t)o.head * D + d0);
      p[0] = make_uint4(r[0], r[1], r[2], r[3]);
      p[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
  } else {
#pragma unroll
    for (int it = 0; it < (D + 127) / 128; ++it) {
      const int d0 = it * 128 + 2 * lane;
      if (d0 >= D) continue;
      uint2 c = make_uint2(zeros, zeros);
      uint4 sv = make_uint4(0, 0, 0, 0);
      if (o.held) {
        c = *reinterpret_cast<const uint2*>(o.base + L.vc + ((o.slot >> 3) * D + d0) * 4);
        sv = *reinterpret_cast<const uint4*>(
            o.base + L.vs + 16 * (((o.slot >> 3) << L.n_shift) + (d0 >> gs)));
      }
      const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
      float x[8], y[8];
      decode8<FMT>(c.x, x);
      decode8<FMT>(c.y, y);
      uint32_t h[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float s = (t & 1) ? bf16_hi(sw[t / 2]) : bf16_lo(sw[t / 2]);
        const bf16x2_t z = {(__bf16)(x[t] * s), (__bf16)(y[t] * s)};
        h[t] = __builtin_bit_cast(uint32_t, z);
      }
      uint16_t* row = a.v_out + (o.row + o.lo) * a.v_stride + (int64_t)o.head * D;
      if (o.lo == 0 && o.hi == 8) {
#pragma unroll
        for (int t = 0; t < 8; ++t, row += a.v_stride)
          *reinterpret_cast<uint32_t*>(row + (uint32_t)d0) = h[t];
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (t >= o.lo && t < o.hi)
            *reinterpret_cast<uint32_t*>(row + (t - o.lo) * a.v_stride + d0) = h[t];
      }
    }
  }
}

// ---- attention ----------------------------------------------------------------------------
// Rows of a tile: row rho of sequence b is (query row rho / r, query head head * r + rho % r) of
// one kv head, so the heads that share keys share a tile.  A wavefront takes 32 positions a step:
//   S^T = K Q^T: A = K (16 positions x 32 d, decoded in place), B = Q^T.  The first matrix holds
//     positions 8 g + 0..3, the second 8 g + 4..7 (g = 0..3), so that lane (q, g) ends up with
//     positions 8 g .. 8 g + 7 of query row q;
//   O^T += V^T P^T: A = V^T (one dword = 8 positions of one d), B = P^T: exactly the 8 values
//     that the lane has.  Nothing passes through LDS or changes lanes.
// Column j of d-tile (c, jj) of V^T is d = 64 c + 4 j + jj: a lane loads 4 d (16 bytes) at once.
//
// Operands are fp16: code value (<= 3 significant bits) times bf16 scale (8) is exact in fp16's
// 11, where bf16 would round it; P enters scaled by 2^P_SHIFT against the running reference, so
// that values down to 2^-18 of the largest keep 11 bits.  Sums, maxima and exponents are fp32.
//
// The reference maximum m moves only when a score passes it by more than MOVE (in powers of 2):
// the steps in between need no exchange between lanes and no rescaling.  P stays below
// 2^(P_SHIFT + MOVE) = 4096, well inside fp16.
constexpr float MOVE = 8.0f;
constexpr float P_SHIFT = 4.0f;

struct Tile {
  Seq s;
  int b, head, rho0, n_rho;  // rows rho0 .. rho0 + n_rho - 1 of this (sequence, head)
  int p_lo, p_hi;            // positions of the first and last row
  int n_steps, sink_steps, main0;  // steps 0 .. sink_steps - 1, then main0, main0 + 1, ...
};
// rho / r for 0 <= rho < 2^30: r_mul = floor(2^32 (2^s - r) / r) + 1, s = ceil(log2 r)
__device__ __forceinline__ int row_of(const Kv4AttnArgs& a, int rho) {
  return (int)((__umulhi((uint32_t)rho, a.r_mul) + (uint32_t)rho) >> a.r_shift);
}
__device__ __forceinline__ bool tile_of(const Kv4AttnArgs& a, const Seq& s, int b, int j, int head,
                                        int R, Tile& t) {
  const int r = a.r;
  t.b = b;
  t.s = s;
  t.head = head;
  t.rho0 = j * R;
  t.n_rho = min(R, t.s.n * r - t.rho0);
  if (j < 0 || t.n_rho <= 0) return false;
  const int first = t.s.len - t.s.n;
  t.p_lo = first + row_of(a, t.rho0);
  t.p_hi = first + row_of(a, t.rho0 + t.n_rho - 1);
  const int end = min(t.p_hi + 1, t.s.cap);  // positions beyond the table hold nothing
  t.n_steps = t.sink_steps = t.main0 = 0;
  if (end > 0) {
    const int last = (end - 1) / KV4_STEP;
    if (a.window > 0 && t.p_lo >= a.window) {
      t.main0 = (t.p_lo - a.window + 1) / KV4_STEP;
      t.sink_steps = min((min(a.sinks, end) + KV4_STEP - 1) / KV4_STEP, min(t.main0, last + 1));
    }
    t.n_steps = t.sink_steps + max(last + 1 - t.main0, 0);
  }
  return true;
}
// Whether the launch is the one that takes this sequence (a call of few and many rows has two).
__device__ __forceinline__ bool takes_seq(const Kv4AttnArgs& a, const Seq& s) {
  return s.n > a.rows_over && s.n <= a.rows_to;
}
__device__ __forceinline__ int position_of(const Tile& t, int step) {
  return (step < t.sink_steps ? step : step - t.sink_steps + t.main0) * KV4_STEP;
}
template <int D>
struct KStage {  // one step's K codes and scales of one lane
  uint32_t c[2][D / 32];
  uint16_t s[2][(D + 127) / 128];
};
template <int D>
struct VStage {
  uint32_t c[D / 16];
  uint4 s[D / 64];
};

template <int D>
struct Offsets {  // per lane, inside a head's part of a page, for position 0
  int kc[2], vc, ks[2][(D + 127) / 128], vs[D / 64];
  __device__ __forceinline__ Offsets(const Kv4Where& w, int lane) {
    const Layout<D> L(w);
    const int m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * (m >> 2) + (m & 3) + 4 * h;
      kc[h] = row * (D / 2) + g * (D == 64 ? 8 : 16);
#pragma unroll
      for (int c = 0; c < (D + 127) / 128; ++c)
        ks[h][c] = L.ks + 2 * ((row << L.n_shift) +
                               ((128 * c + g * (D == 64 ? 16 : 32)) >> w.group_shift));
    }
    vc = L.vc + (g * D + 4 * m) * 4;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      vs[c] = L.vs + 16 * ((g << L.n_shift) + ((64 * c + 4 * m) >> w.group_shift));
  }
};

// Where a step's 32 positions lie: the head's part of their page, and the byte offsets of the
// step's codes and scales in it.
struct Place {
  const uint8_t* codes;
  const uint8_t* scales;
};
template <int D>
__device__ __forceinline__ Place place_of(const Kv4Where& w, int head, int page, int t0) {
  const int in_page = t0 & ((1 << w.page_shift) - 1);
  const int n_shift = (D == 64 ? 6 : D == 128 ? 7 : 8) - w.group_shift;
  const uint8_t* base = w.cache + page * w.page_bytes + (int64_t)head * w.head_bytes;
  return {base + in_page * (D / 2), base + ((in_page << n_shift) << 1)};
}
template <int D>
__device__ __forceinline__ void load_k(const Place& p, const Offsets<D>& off, KStage<D>& x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (D == 64) {
      const uint2 c = *reinterpret_cast<const uint2*>(p.codes + off.kc[h]);
      x.c[h][0] = c.x;
      x.c[h][1] = c.y;
    } else {
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        const uint4 u = *reinterpret_cast<const uint4*>(p.codes + off.kc[h] + 64 * c);
        x.c[h][4 * c] = u.x; x.c[h][4 * c + 1] = u.y;
        x.c[h][4 * c + 2] = u.z; x.c[h][4 * c + 3] = u.w;
      }
    }
#pragma unroll
    for (int c = 0; c < (D + 127) / 128; ++c)
      x.s[h][c] = *reinterpret_cast<const uint16_t*>(p.scales + off.ks[h][c]);
  }
}
template <int D>
__device__ __forceinline__ void load_v(const Place& p, const Offsets<D>& off, VStage<D>& x) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const uint4 u = *reinterpret_cast<const uint4*>(p.codes + off.vc + 256 * c);
    x.c[4 * c] = u.x; x.c[4 * c + 1] = u.y; x.c[4 * c + 2] = u.z; x.c[4 * c + 3] = u.w;
    x.s[c] = *reinterpret_cast<const uint4*>(p.scales + off.vs[c]);
  }
}

// Dword of 8 codes -> 8 fp16 values times the scales.  INT4: a nibble moved to mantissa bits
// 6 .. 9 under the exponent of 16 reads as 16 + n; (16 + n) s - 24 s is one fma, exact because
// 24 s is (3 more bits than s).  It leaves the pairs (0, 4), (1, 5), (2, 6), (3, 7): Q, P and the V
// scales are laid out in that order.  FP4: the hardware's conversion, pairs (0, 1) .. (6, 7).
template <int FMT>
__device__ __forceinline__ f16x8_t decode_f16(uint32_t w, const f16x2_t (&s)[4],
                                              const f16x2_t (&s24)[4]) {
  f16x2_t p[4];
  if constexpr (FMT == FMT_INT4) {
    // (the mask in a vector and the exponent in a scalar register: and_or takes them as one
    // instruction, where two literals make it two)
    uint32_t mask = 0x03C003C0u, sixteen = 0x4C004C00u;
    asm("" : "+v"(mask));
    asm("" : "+s"(sixteen));
    const uint32_t u[4] = {w << 6, w << 2, w >> 2, w >> 6};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, (u[i] & mask) | sixteen), s[i],
                                       s24[i]);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s[0];
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s[1];
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s[2];
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s[3];
  }
  struct { f16x2_t p[4]; } r = {{p[0], p[1], p[2], p[3]}};
  return __builtin_bit_cast(f16x8_t, r);
}
// index of the value that operand half i holds
template <int FMT>
__host__ __device__ constexpr int value_at(int i) {
  return FMT == FMT_INT4 ? (i >> 1) + 4 * (i & 1) : i;
}

// Query rows of one (sequence, head): lane (q, g) holds row q of each 16-row tile as the B operand
// of S^T, the d of K dword i in that dword's value order, and its row's position.
template <int D, int NT>
struct Queries {
  f16x8_t q[NT][D / 32];
  int pos[NT];
};
template <int D, int NT>
__device__ __forceinline__ void load_queries(const Kv4AttnArgs& a, const Tile& t, int q16, int g,
                                             uint4 (&u)[NT][D / 32], int (&pos)[NT]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rho = t.rho0 + 16 * nt + q16;
    const bool on = 16 * nt + q16 < t.n_rho;
    const int i = row_of(a, rho), h = t.head * a.r + rho - i * a.r;
    pos[nt] = on ? t.s.len - t.s.n + i : -1;
    const uint16_t* p = a.q + (int64_t)(t.s.row0 + i) * a.q_stride + (int64_t)h * D;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const int d0 = D == 64 ? 16 * g + 8 * j : 128 * (j / 4) + 32 * g + 8 * (j % 4);
      u[nt][j] = make_uint4(0, 0, 0, 0);
      if (on) u[nt][j] = *reinterpret_cast<const uint4*>(p + d0);
    }
  }
}
template <int D, int FMT, int NT>
__device__ __forceinline__ void convert_queries(const uint4 (&u)[NT][D / 32], Queries<D, NT>& x) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const uint32_t uw[4] = {u[nt][j].x, u[nt][j].y, u[nt][j].z, u[nt][j].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = value_at<FMT>(e);
        x.q[nt][j][e] = (_Float16)((d & 1) ? bf16_hi(uw[d / 2]) : bf16_lo(uw[d / 2]));
      }
    }
}

template <int D, int NT>
struct Acc {
  f32x4_t o[NT][D / 64][4];
  float m[NT], l[NT];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -FLT_MAX;
      l[nt] = 0.0f;
#pragma unroll
      for (int e = 0; e < D / 64; ++e)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) o[nt][e][jj] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }
};

// Scores of a step's 32 positions, in powers of 2.
template <int D, int FMT, int NT>
__device__ __forceinline__ void step_scores(const KStage<D>& x, const Queries<D, NT>& q, float c,
                                            f32x4_t (&sc)[NT][2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const _Float16 s1 = (_Float16)bf16_to_f32(x.s[h][D == 64 ? 0 : i / 4]);
      const f16x2_t s = {s1, s1};
      const f16x2_t s24 = s * (f16x2_t){(_Float16)-24.0f, (_Float16)-24.0f};
      const f16x2_t s4[4] = {s, s, s, s}, z4[4] = {s24, s24, s24, s24};
      const f16x8_t k = decode_f16<FMT>(x.c[h][i], s4, z4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        sc[nt][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q.q[nt][i], sc[nt][h], 0, 0, 0);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) sc[nt][h] *= c;
}

// largest scale whose values and decode constants (INT4: 24 s) are finite in fp16, as bf16 bits
__host__ __device__ constexpr uint32_t scale_limit(int fmt) {
  return fmt == FMT_INT4 ? 0x452Au : 0x462Au;
}

// Steps with positions that some row does not see.  What lies there may be anything: scores are
// replaced and V scales cleared.  A position whose V scale fp16 cannot take and that only some rows
// see is cleared too, and the rows that see it get a NaN score.
template <int D, int FMT, int NT>
__device__ __forceinline__ void step_mask(const Kv4AttnArgs& a, const Tile& t, int t0, int g,
                                          const Queries<D, NT>& q, f32x4_t (&sc)[NT][2],
                                          uint4 (&vs)[D / 64]) {
  uint32_t vw[D / 64][4];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    vw[e][0] = vs[e].x; vw[e][1] = vs[e].y; vw[e][2] = vs[e].z; vw[e][3] = vs[e].w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = t0 + 8 * g + i;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      const uint32_t b16 = (i & 1) ? vw[e][i / 2] >> 16 : vw[e][i / 2] & 0xFFFFu;
      bad |= (b16 & 0x7FFFu) > scale_limit(FMT);
    }
    const uint64_t bads = __ballot(bad);
    const bool poisoned = ((bads >> (16 * g)) & 0xFFFFu) != 0;
    if (poisoned || p > t.p_hi)
#pragma unroll
      for (int e = 0; e < D / 64; ++e) vw[e][i / 2] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool seen = p <= q.pos[nt] &&
                        (a.window == 0 || p > q.pos[nt] - a.window || p < a.sinks);
      const float s = sc[nt][i >> 2][i & 3];
      sc[nt][i >> 2][i & 3] = !seen ? -INFINITY : poisoned ? NAN : s;
    }
  }
#pragma unroll
  for (int e = 0; e < D / 64; ++e) vs[e] = make_uint4(vw[e][0], vw[e][1], vw[e][2], vw[e][3]);
}
__device__ __forceinline__ bool step_at_edge(const Kv4AttnArgs& a, const Tile& t, int t0) {
  return t0 + KV4_STEP - 1 > t.p_lo ||
         (a.window > 0 && t0 <= t.p_hi - a.window && t0 + KV4_STEP > a.sinks);
}

// Scores -> weights: the reference maximum moves where a score passes it by more than MOVE.
template <int D, int FMT, int NT>
__device__ __forceinline__ void step_weights(const f32x4_t (&sc)[NT][2], Acc<D, NT>& acc,
                                             f16x8_t (&p)[NT]) {
  bool move = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mx = sc[nt][0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, sc[nt][i >> 2][i & 3]);
    move |= mx > acc.m[nt] + MOVE;
  }
  if (__ballot(move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx = acc.m[nt];
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, sc[nt][i >> 2][i & 3]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float f = __builtin_amdgcn_exp2f(acc.m[nt] - mx);
      acc.m[nt] = mx;
      acc.l[nt] *= f;
#pragma unroll
      for (int e = 0; e < D / 64; ++e)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) acc.o[nt][e][jj] *= f;
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float ref = acc.m[nt] - P_SHIFT;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_exp2f(sc[nt][i >> 2][i & 3] - ref);
    acc.l[nt] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
#pragma unroll
    for (int i = 0; i < 8; ++i) p[nt][i] = (_Float16)v[value_at<FMT>(i)];
  }
}

// O^T += V^T P^T
template <int D, int FMT, int NT>
__device__ __forceinline__ void step_values(const VStage<D>& x, const f16x8_t (&p)[NT],
                                            Acc<D, NT>& acc) {
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const uint32_t w[4] = {x.s[e].x, x.s[e].y, x.s[e].z, x.s[e].w};
    f16x2_t s[4], s24[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int i0 = value_at<FMT>(2 * i), i1 = value_at<FMT>(2 * i + 1);
      s[i] = f16x2_t{(_Float16)((i0 & 1) ? bf16_hi(w[i0 / 2]) : bf16_lo(w[i0 / 2])),
                     (_Float16)((i1 & 1) ? bf16_hi(w[i1 / 2]) : bf16_lo(w[i1 / 2]))};
      s24[i] = s[i] * (f16x2_t){(_Float16)-24.0f, (_Float16)-24.0f};
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const f16x8_t v = decode_f16<FMT>(x.c[4 * e + jj], s, s24);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        acc.o[nt][e][jj] =
            __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[nt], acc.o[nt][e][jj], 0, 0, 0);
    }
  }
}

// One row of the result: o = sum / l (zero where nothing was visible), lse = ln(sum of exp).
__device__ __forceinline__ float row_inv(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.0f || l != l ? (m - P_SHIFT) * LN2 + logf(l) : -INFINITY;
}

// ---- pieces -------------------------------------------------------------------------------
// A workgroup takes one piece: the steps of a row tile, or where there are more workgroups than
// tiles an equal part of them.  `per` steps a piece are chosen on the device, from the batch's
// actual lengths, as the fewest for which the pieces are no more than the workgroups that run at
// once (or than the tiles), so that ragged batches, single long caches and many short ones load
// the GPU evenly in one round.  (Cutting the steps of all tiles, end to end, into equal parts
// loads it more evenly still, but parts that reach over two tiles pay a workgroup's start and end
// twice, 8 us: 8 sequences of up to 4099 positions and 4 rows took 28 us that way and take 20, 32
// of up to 8192 took 31 and take 30.)
// The pieces of a cut tile leave partial sums, and the workgroup that finishes last joins them in
// order of position.
// Tiles of a sequence and (an upper bound of) the steps of each; a tile that sees nothing counts
// one step, so that its rows are written.
__device__ __forceinline__ void seq_work(const Kv4AttnArgs& a, const Seq& s, int R, int* tiles,
                                         int* steps) {
  *tiles = takes_seq(a, s) ? (int)(((int64_t)s.n * a.r + R - 1) / R) : 0;
  const int end = min(s.len, s.cap);
  int w = (end + KV4_STEP - 1) / KV4_STEP;
  if (a.window > 0) {
    const int rows = (R + a.r - 2) / a.r + 1;  // rows of a tile, at most
    const int main = (a.window - 1 + rows + 2 * KV4_STEP - 2) / KV4_STEP;
    const int first = (min(a.sinks, end) + KV4_STEP - 1) / KV4_STEP;
    if (main + first > 0) w = min(w, main + first);
  }
  *steps = max(w, 1);
}
// Pieces of a tile of `steps` steps, of *chunk steps each; the last may be shorter.
__device__ __forceinline__ int cut_steps(const Kv4AttnArgs& a, int steps, int per, int* chunk) {
  *chunk = steps;
  if (steps <= per || steps <= 2 * a.min_steps) return 1;
  const unsigned k = ((unsigned)steps + per - 1) / (unsigned)per;
  // multiples of 8: a step more costs a wavefront of 8 as much as 8
  *chunk = (int)(((unsigned)steps + k - 1) / k + 7) & ~7;
  return (int)(((unsigned)steps + *chunk - 1) / (unsigned)*chunk);
}
__device__ __forceinline__ int wave_total(int v) {
  return __builtin_amdgcn_readlane(wave_incl_sum(v), 63);
}

struct Piece {
  Seq s;
  int b, tile;     // sequence, and its tile
  int s0, s1;      // steps of the tile
  int n, index;    // pieces of the tile, and which of them this is
  int partial;     // where its partial sums go, in units of partials
};
// at: the piece's place among those of sequence f.b, which has `tiles` tiles cut into f.n pieces
__device__ __forceinline__ bool set_piece(const Kv4AttnArgs& a, int at, int tiles, int steps,
                                          int chunk, Piece& f) {
  f.tile = f.n > 1 ? at / f.n : at;
  f.index = at - f.tile * f.n;
  f.s0 = f.index * chunk;
  f.s1 = min(f.s0 + chunk, steps);
  // (always so for cu_rows that ascend)
  const int first = f.partial - f.index;
  return f.tile >= 0 && f.tile < tiles &&
         (f.n == 1 || (first >= 0 && first <= 2 * a.n_parts - f.n));
}
// The x-th piece, from the last (the pieces of later tiles, which see more, first); false: there
// are not as many.  Uniform over the workgroup.
// Up to 64 sequences: one a lane.  More: from the plan that a kernel before this one has made (as
// many loads as a search needs; every workgroup going through the whole batch took 7.5 ms where
// 4096 single tokens of 8 kv heads take 0.8), or, where nothing is cut, by slots:
// floor(cu[b + 1] r / R) - floor(cu[b] r / R) + 1 are enough for the tiles of sequence b.
__device__ __forceinline__ bool find_piece(const Kv4AttnArgs& a, int R, int x, Piece& f) {
  int tiles, steps, chunk;
  if (a.w.B > 64) {
    int at;
    if (a.plan) {
      const int2 all = a.plan[a.w.B];
      x = all.x - 1 - x;
      if (x < 0) return false;
      f.b = last_at_most(a.w.B, x, [&](int b) { return a.plan[b].x; });
      const int2 before = a.plan[f.b];
      f.s = seq_at(a.w, f.b);
      seq_work(a, f.s, R, &tiles, &steps);
      f.n = cut_steps(a, steps, all.y, &chunk);
      at = x - before.x;
      f.partial = before.y + at;
    } else {
      const auto slots = [&](int c) { return c * a.r / R; };
      x = a.n_groups - 1 - x;
      f.b = seq_of_slot(a.w, x, 1, slots);
      f.s = seq_at(a.w, f.b);
      seq_work(a, f.s, R, &tiles, &steps);
      f.n = 1;
      chunk = steps;
      at = x - (slots(f.s.row0) + f.b);
      f.partial = 0;
    }
    return set_piece(a, at, tiles, steps, chunk, f);
  }
  const int b = threadIdx.x & 63;
  Seq s{0, 0, 0, 0};
  tiles = 0;
  steps = 1;
  if (b < a.w.B) {
    s = seq_at(a.w, b);
    seq_work(a, s, R, &tiles, &steps);
  }
  int per = 1 << 30;
  if (a.part) {
    const int most = max(a.n_parts, wave_total(tiles));
    per = max((wave_total(tiles * steps) + a.n_parts - 1) / a.n_parts, a.min_steps);
    while (true) {
      const float r = __builtin_amdgcn_rcpf((float)per);
      if (wave_total(tiles * max((int)ceilf((float)steps * r - 1e-3f), 1)) <= most) break;
      per += (per >> 3) + 1;
    }
  }
  const int k = cut_steps(a, steps, per, &chunk), mine = tiles * k, cut = k > 1 ? mine : 0;
  const int incl = wave_incl_sum(mine), cincl = wave_incl_sum(cut);
  x = __builtin_amdgcn_readlane(incl, 63) - 1 - x;
  if (x < 0) return false;
  f.b = min(__popcll(__ballot(incl <= x)), 63);
  const int at = x - __builtin_amdgcn_readlane(incl - mine, f.b);
  f.n = __builtin_amdgcn_readlane(k, f.b);
  f.partial = __builtin_amdgcn_readlane(cincl - cut, f.b) + at;
  f.s.row0 = __builtin_amdgcn_readlane(s.row0, f.b);
  f.s.n = __builtin_amdgcn_readlane(s.n, f.b);
  f.s.len = __builtin_amdgcn_readlane(s.len, f.b);
  f.s.cap = __builtin_amdgcn_readlane(s.cap, f.b);
  return set_piece(a, at, __builtin_amdgcn_readlane(tiles, f.b),
                   __builtin_amdgcn_readlane(steps, f.b), __builtin_amdgcn_readlane(chunk, f.b), f);
}

// The plan of a batch of more than 64 sequences: for each the pieces, and the pieces of cut tiles,
// before its own; behind them all pieces, and the steps of a piece.  One workgroup.
constexpr int PLAN_THREADS = 1024;
__global__ __launch_bounds__(PLAN_THREADS) void kv4_plan_kernel(Kv4AttnArgs a, int R) {
  __shared__ int sums[2][PLAN_THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // sums over the threads before this one, and over all
  const auto scan = [&](int x, int y, int2& before, int2& all) {
    const int ix = wave_incl_sum(x), iy = wave_incl_sum(y);
    __syncthreads();
    if (lane == 63) {
      sums[0][wave] = ix;
      sums[1][wave] = iy;
    }
    __syncthreads();
    before = make_int2(ix - x, iy - y);
    all = make_int2(0, 0);
    for (int w = 0; w < PLAN_THREADS / 64; ++w) {
      before.x += w < wave ? sums[0][w] : 0;
      before.y += w < wave ? sums[1][w] : 0;
      all.x += sums[0][w];
      all.y += sums[1][w];
    }
  };
  int total = 0, tiles, steps, chunk;
  for (int b = tid; b < a.w.B; b += PLAN_THREADS) {
    seq_work(a, seq_at(a.w, b), R, &tiles, &steps);
    total += tiles * steps;
  }
  int2 before, all, done = make_int2(0, 0);
  scan(total, 0, before, all);
  const int per = max((all.x + a.n_parts - 1) / a.n_parts, a.min_steps);
  for (int b0 = 0; b0 < a.w.B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    int mine = 0, cut = 0;
    if (b < a.w.B) {
      seq_work(a, seq_at(a.w, b), R, &tiles, &steps);
      const int k = cut_steps(a, steps, per, &chunk);
      mine = tiles * k;
      cut = k > 1 ? mine : 0;
    }
    scan(mine, cut, before, all);
    if (b < a.w.B) a.plan[b] = make_int2(done.x + before.x, done.y + before.y);
    done.x += all.x;
    done.y += all.y;
  }
  if (tid == 0) a.plan[a.w.B] = make_int2(done.x, per);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_rsrc(const float* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), 0, 0x7FFFFFFF, 0x00020000);
}
// 16-byte accesses that other workgroups of the launch see (sc1: past the XCD's L2)
__device__ __forceinline__ void st4_agent(__amdgpu_buffer_rsrc_t r, int word, float4 v) {
  const u32x4_t d = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                     __float_as_uint(v.w)};
  __builtin_amdgcn_raw_buffer_store_b128(d, r, word * 4, 0, 16);
}
__device__ __forceinline__ float4 ld4_agent(__amdgpu_buffer_rsrc_t r, int word) {
  const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(r, word * 4, 0, 16);
  return make_float4(__uint_as_float(d.x), __uint_as_float(d.y), __uint_as_float(d.z),
                     __uint_as_float(d.w));
}

// Output of 4 columns of one row.
__device__ __forceinline__ void store_out4(const Kv4AttnArgs& a, const Tile& t, int D, int row, int d,
                                           float4 v, float inv) {
  const int rho = t.rho0 + row, i = row_of(a, rho), qi = t.s.row0 + i;
  const int h = t.head * a.r + rho - i * a.r;
  const bf16x2_t lo = {(__bf16)(v.x * inv), (__bf16)(v.y * inv)};
  const bf16x2_t hi = {(__bf16)(v.z * inv), (__bf16)(v.w * inv)};
  *reinterpret_cast<uint2*>(a.out + (int64_t)qi * a.out_stride + (int64_t)h * D + d) =
      make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}
__device__ __forceinline__ void store_lse(const Kv4AttnArgs& a, const Tile& t, int row, float m,
                                          float l) {
  const int rho = t.rho0 + row, i = row_of(a, rho), qi = t.s.row0 + i;
  const int h = t.head * a.r + rho - i * a.r;
  if (a.lse) a.lse[(int64_t)qi * a.Hq + h] = row_lse(m, l);
}

// Joins the n partials of one tile, from `first` on.  A wavefront takes a row at a time; LR lanes
// hold a row, so it reads 64 / LR partials at once.
template <int D, int R>
__device__ __forceinline__ void join_parts(const Kv4AttnArgs& a, const Tile& t, int first, int n,
                                           int wave, int n_waves) {
  constexpr int LR = D / 4, PL = 64 / LR, SIZE = R * (D + 2);
  const int lane = threadIdx.x & 63, sub = lane / LR, d = 4 * (lane % LR);
  const __amdgpu_buffer_rsrc_t r = part_rsrc(a.part);
  for (int row = wave; row < t.n_rho; row += n_waves) {
    float m = -FLT_MAX, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = 0; k0 < n; k0 += 64) {
      const int k = min(k0 + lane, n - 1);
      const int here = min(n - k0, 64);
      const int at = (first + k) * SIZE + R * D + row;
      float pm = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at * 4, 0, 16));
      float pl = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (at + R) * 4, 0, 16));
      float f = 0.0f;
      constexpr int UN = 16;  // loads in flight
      for (int j0 = 0; j0 < here; j0 += UN * PL) {
        float4 v[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const int kk = k0 + min(j0 + u * PL + sub, here - 1);
          v[u] = ld4_agent(r, (first + kk) * SIZE + row * D + d);
        }
        if (j0 == 0) {  // the chunk's weights, while the first sums are on their way
          if (lane >= here) {
            pm = -FLT_MAX;
            pl = 0.0f;
          }
          float mx = pm;
#pragma unroll
          for (int i = 1; i < 64; i *= 2) mx = fmaxf(mx, __shfl_xor(mx, i));
          mx = fmaxf(mx, m);
          const float f0 = __builtin_amdgcn_exp2f(m - mx);
          m = mx;
          f = __builtin_amdgcn_exp2f(pm - m);
          l = l * f0 + f * pl;
          o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const int j = j0 + u * PL + sub;
          float fk = __shfl(f, min(j, here - 1));  // (every lane takes part)
          fk = j < here ? fk : 0.0f;
          o.x += fk * v[u].x; o.y += fk * v[u].y; o.z += fk * v[u].z; o.w += fk * v[u].w;
        }
      }
    }
#pragma unroll
    for (int i = 1; i < 64; i *= 2) l += __shfl_xor(l, i);
#pragma unroll
    for (int i = LR; i < 64; i *= 2) {
      o.x += __shfl_xor(o.x, i); o.y += __shfl_xor(o.y, i);
      o.z += __shfl_xor(o.z, i); o.w += __shfl_xor(o.w, i);
    }
    if (sub == 0) store_out4(a, t, D, row, d, o, row_inv(l));
    if (lane == 0) store_lse(a, t, row, m, l);
  }
}

// ---- attention of few rows over long caches -------------------------------------------------
// NW (4 or 8) wavefronts take a piece's steps of 32 positions in turn and join their sums through
// LDS; codes go from memory to registers to matrix operands, each read once.  The next step's codes
// are loaded behind the arithmetic of this one (two steps ahead gained nothing, 128 registers for
// 4 wavefronts a SIMD spilled).
// Measured: a single cache of 131072 positions, 4 kv heads of 128: 23 us, of which the loop takes
// 13 at 5.8 TB/s; the rest is a workgroup's chain of dependent steps: start 2 to 4 us (workgroups
// are started one after the other), finding its piece 2, table and first codes 1.3, joining
// wavefronts 2, joining 64 parts 4.  A batch of 32 such heads' caches of up to 8192: 30 us (97 MB);
// 1000 positions of one sequence: 10 us, all of it that chain.
template <int D, int FMT, int NT, int NW>
__global__ __launch_bounds__(64 * NW, 2) void kv4_attn_rows_kernel(Kv4AttnArgs a) {
  constexpr int R = 16 * NT, LD = D + 4, SIZE = R * (D + 2);
  __shared__ float lds_o[NW][16][LD];
  __shared__ float lds_m[NW][R], lds_l[NW][R];
  __shared__ int lds_flag;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q16 = lane & 15, g = lane >> 4;
  const int head = blockIdx.x % a.w.Hkv;
  Piece f;
  if (!find_piece(a, R, blockIdx.x / a.w.Hkv, f)) return;
  Tile t;
  tile_of(a, f.s, f.b, f.tile, head, R, t);
  const int s0 = f.s0;
  const bool whole = f.n == 1;
  const float c = a.scale * LOG2E;
  const Offsets<D> off(a.w, lane);
  if (t.s.len > t.s.cap && s0 == 0 && threadIdx.x == 0) report(a.w.status, ST_LENGTH);
  Acc<D, NT> acc;
  acc.clear();
  bool all_ok = true;
  const int last = min(f.s1, t.n_steps);
  uint4 raw[NT][D / 32];
  Queries<D, NT> q;
  bool first_round = true;
  for (int base = s0 + wave; base < last; base += 64 * NW) {
    // pages of up to 64 of the wavefront's steps, one a lane; -1: no such page
    int pages;
    {
      const int step = min(base + lane * NW, last - 1);
      pages = a.w.table[(int64_t)t.b * a.w.max_pages + (position_of(t, step) >> a.w.page_shift)];
    }
    if (first_round) load_queries<D, NT>(a, t, q16, g, raw, q.pos);
    if (pages < 0 || pages >= a.w.num_pages) pages = -1;
    const int n = min((last - base + NW - 1) / NW, 64);
    KStage<D> ks;
    VStage<D> vs;
    int t0 = position_of(t, base), page = __builtin_amdgcn_readlane(pages, 0);
    Place pl = place_of<D>(a.w, head, max(page, 0), t0);
    load_k<D>(pl, off, ks);
    load_v<D>(pl, off, vs);
    if (first_round) convert_queries<D, FMT, NT>(raw, q);
    first_round = false;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      // the wavefronts of a SIMD go first in turn: left alone, the older one always does, and the
      // other ends 4 us behind it (wavefronts of several workgroups: 3 to 5 % in all)
      if ((i ^ (wave >> 2)) & 1)
        __builtin_amdgcn_s_setprio(1);
      else
        __builtin_amdgcn_s_setprio(0);
      if (page >= 0) {
        f32x4_t sc[NT][2];
        step_scores<D, FMT, NT>(ks, q, c, sc);
        if (step_at_edge(a, t, t0)) step_mask<D, FMT, NT>(a, t, t0, g, q, sc, vs.s);
        f16x8_t p[NT];
        step_weights<D, FMT, NT>(sc, acc, p);
        step_values<D, FMT, NT>(vs, p, acc);
      } else {
        all_ok = false;
      }
      if (i + 1 < n) {
        t0 = position_of(t, base + (i + 1) * NW);
        page = __builtin_amdgcn_readlane(pages, i + 1);
        pl = place_of<D>(a.w, head, max(page, 0), t0);
        load_k<D>(pl, off, ks);
        load_v<D>(pl, off, vs);
      }
    }
  }
  if (!all_ok && lane == 0) report(a.w.status, ST_PAGE);

  // join the wavefronts: sums to LDS, then each wavefront adds every 8th row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float l = acc.l[nt];
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
      lds_m[wave][16 * nt + q16] = acc.m[nt];
      lds_l[wave][16 * nt + q16] = l;
    }
  }
  const int partial = head * 2 * a.n_parts + f.partial;
  const __amdgpu_buffer_rsrc_t pr = part_rsrc(a.part);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (nt > 0) __syncthreads();
    float* dst = &lds_o[wave][q16][0];
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(dst + 64 * e + 16 * g + 4 * i) =
            make_float4(acc.o[nt][e][0][i], acc.o[nt][e][1][i], acc.o[nt][e][2][i],
                        acc.o[nt][e][3][i]);
    __syncthreads();
#pragma unroll
    for (int rr = 0; rr < 16 / NW; ++rr) {
      const int row16 = wave + NW * rr, row = 16 * nt + row16;
      if (row < t.n_rho) {
        float m = lds_m[0][row];
#pragma unroll
        for (int w = 1; w < NW; ++w) m = fmaxf(m, lds_m[w][row]);
        float l = 0.0f, f[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          f[w] = __builtin_amdgcn_exp2f(lds_m[w][row] - m);
          l += lds_l[w][row] * f[w];
        }
        const int d = 4 * lane;
        if (d < D) {
          float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const float4 z = *reinterpret_cast<const float4*>(&lds_o[w][row16][d]);
            u.x += f[w] * z.x; u.y += f[w] * z.y; u.z += f[w] * z.z; u.w += f[w] * z.w;
          }
          if (whole)
            store_out4(a, t, D, row, d, u, row_inv(l));
          else
            st4_agent(pr, partial * SIZE + row * D + d, u);
        }
        if (lane == 0) {
          if (whole) {
            store_lse(a, t, row, m, l);
          } else {
            st_sc1(a.part, (size_t)partial * SIZE + R * D + row, m);
            st_sc1(a.part, (size_t)partial * SIZE + R * D + R + row, l);
          }
        }
      }
    }
  }
  if (!whole) {
    unsigned* counter = a.counters + head * 2 * a.n_parts + (f.partial - f.index);
    if (last_arriver(counter, (unsigned)f.n, &lds_flag)) {
      join_parts<D, R>(a, t, partial - f.index, f.n, wave, NW);
      if (threadIdx.x == 0) st_cnt(counter, 0u);
    }
  }
}

// ---- attention of many rows -------------------------------------------------------------------
// A workgroup of 8 wavefronts walks the visible positions 64 at a time (a turn).  The codes are
// decoded once for all its rows, into LDS:
//   K: [D / 8][64] units of 16 bytes (8 d of one position; see k_unit), V: [8][D] units (8 positions
//   of one d).  Both are the A operands of 32x32x16 matrix instructions as they lie.
//   S^T = K Q^T, O^T += V^T P^T as above; row m of a 32-position A operand is position
//   16 (m / 16) + 8 ((m / 4) % 2) + 4 ((m % 16) / 8) + m % 4, so that lane (q, h) ends up with
//   positions 16 k + 8 h .. + 7 of row q in registers 8 k .. 8 k + 7: the B operand of O^T.
// D <= 128: a wavefront holds 32 rows whole.  D = 256: two wavefronts hold 32 rows; each takes
// half of a turn's positions for S and half of the columns of O, whose sums would not fit
// otherwise, and they trade row maxima and weights through LDS.
//
// Wavefronts 0-3 (group 0) and 4-7 (group 1), one of each on every SIMD, do a turn's work in
// different orders, so that one has matrix instructions while the other has arithmetic.
// D <= 128, one barrier a turn (two buffers of K and of V): group 0 takes scores, weights, outputs,
// decoding of the next turn; group 1 starts with the decoding.  Weights with outputs, and group 1's
// decoding, go before the other wavefront's instructions (causal prompts of 2 times 4096 rows: 252
// us; 272 without, and with either of the two alone).
// D = 256: two phases with a barrier behind each: M, the matrix instructions (S of this turn, O of
// the turn before), and A, the arithmetic (weights of this turn, decoding).  Slot 2 t (between two
// barriers) is phase M of turn t for group 0 and phase A of turn t - 1 for group 1, slot 2 t + 1 the
// other way round; the phases A of both slots decode K of turn t + 1 and V of turn t, each thread
// its share.  (K of turn t + 1 takes the place of turn t - 1's, last read in slot 2 t - 1, and is
// first read in slot 2 t + 2; V of turn t that of turn t - 2's, last read in slot 2 t - 1, first
// read in slot 2 t + 2.)
//
// Bound by matrix instructions together with the arithmetic between them (a SIMD overlaps the two of
// different wavefronts only in part): two causal prompts of 4096 rows, 32 heads of 128, 220 us in a
// row (870 TFLOP/s; a large matrix product reaches 1150), 250 after other work; a prompt of 8192
// rows, 16 heads of 256, window 1024, 210 us (615 TFLOP/s).  Interleaving the two kinds by hand in one
// wavefront spilled and took 373 us; the two phases of D = 256 took 305 for heads of 128.
constexpr int TILE_POS = 64, TILE_THREADS = 512;
// where the units of 8 d's positions start: those that 8 threads write at once (D / 64 rows of
// units apart) lie 1 or 2 units apart modulo the 16 that the banks hold, so that a wavefront's units
// spread.  (256: rows 65 apart put them on 4 of the 16; 128: 2 padding units for 2 rows took 1 to
// 3 % longer.)
__host__ __device__ constexpr int k_unit(int D, int u) {
  return TILE_POS * u + (D > 128 ? 2 * (u / 4) : u);
}
__host__ __device__ constexpr int tile_halves(int D) { return D > 128 ? 2 : 1; }
__host__ __device__ constexpr int tile_rows(int D) { return 16 * kv4_tile_nt(D); }
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// halves of a dword of V scales that are above the limit, as nonzero halves
template <int FMT>
__device__ __forceinline__ uint32_t above_limit(uint32_t w) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 lim = {(unsigned short)scale_limit(FMT), (unsigned short)scale_limit(FMT)};
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, w & 0x7FFF7FFFu), lim));
}

template <int D>
struct TileStage {  // one thread's codes and scales: K and V scales of a turn, V of the one before
  static constexpr int N = D / 64, NE = (D + 127) / 128;  // dwords of K, and of V
  uint32_t k[N], v[N];
  uint16_t ks;
  uint4 vs[NE];
};
// Thread -> codes: K: position tid / 8, N consecutive dwords (one scale); V: the wavefront's block
// of 8 positions, its i-th d at vd + v_step(i): two of every 128 columns, in one scale group.
__host__ __device__ constexpr int v_step(int i) { return 16 * (i & 1) + 128 * (i >> 1); }
template <int D>
struct TileMap {
  int tok, kd, blk, vd;
  __device__ __forceinline__ TileMap(int tid) {
    const int lane = tid & 63;
    tok = tid >> 3;
    kd = (tid & 7) * (D / 64);
    blk = tid >> 6;
    vd = D == 64 ? lane : (lane >> 4) * 32 + (lane & 15);
  }
};
// A thread's byte offsets from a step's codes: its own are constant, the scales lie `scales` away.
template <int D>
struct TileOffsets {
  uint32_t kc, vc, ks, vs[TileStage<D>::NE];
  __device__ __forceinline__ TileOffsets(const Kv4Where& w, const Layout<D>& L, const TileMap<D>& m) {
    const int tok = m.tok & (KV4_STEP - 1), blk = m.blk & 3;
    kc = tok * (D / 2) + 4 * m.kd;
    vc = L.vc + (blk * D + m.vd) * 4;
    ks = L.ks + 2 * ((tok << L.n_shift) + ((8 * m.kd) >> w.group_shift));
#pragma unroll
    for (int e = 0; e < TileStage<D>::NE; ++e)
      vs[e] = L.vs + 16 * ((blk << L.n_shift) + ((m.vd + 128 * e) >> w.group_shift));
  }
};
template <class T>
__device__ __forceinline__ T load_at(const uint8_t* base, uint32_t off) {
  return *reinterpret_cast<const T*>(base + off);
}
template <int D>
__device__ __forceinline__ void tile_load_k(const uint8_t* codes, uint32_t scales,
                                            const TileOffsets<D>& off, TileStage<D>& x) {
  if constexpr (D == 64) {
    x.k[0] = load_at<uint32_t>(codes, off.kc);
  } else if constexpr (D == 128) {
    const uint2 u = load_at<uint2>(codes, off.kc);
    x.k[0] = u.x; x.k[1] = u.y;
  } else {
    const uint4 u = load_at<uint4>(codes, off.kc);
    x.k[0] = u.x; x.k[1] = u.y; x.k[2] = u.z; x.k[3] = u.w;
  }
  x.ks = load_at<uint16_t>(codes, off.ks + scales);
#pragma unroll
  for (int e = 0; e < TileStage<D>::NE; ++e) x.vs[e] = load_at<uint4>(codes, off.vs[e] + scales);
}
template <int D>
__device__ __forceinline__ void tile_load_v(const uint8_t* codes, const TileOffsets<D>& off,
                                            TileStage<D>& x) {
#pragma unroll
  for (int i = 0; i < TileStage<D>::N; ++i) x.v[i] = load_at<uint32_t>(codes, off.vc + 4 * v_step(i));
}

// Keeps the order of what is written on both sides: left alone, the compiler reads one operand from
// LDS, waits for it, multiplies and reads the next into the same registers.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// S^T of NU times 32 positions; k: the lane's unit of the first operand.  Four operands are read
// while the four before them are multiplied.
template <int D, int NU>
__device__ __forceinline__ void tile_scores(const uint4* k, const f16x8_t (&q)[D / 16],
                                            f32x16_t (&sc)[NU]) {
  constexpr int J = 4 / NU, G = D / 16 / J;  // groups of 4 operands: J times 16 d
  const auto read = [&](int n, uint4 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = k[k_unit(D, 2 * (J * n + i / NU)) + 32 * (i % NU)];
  };
  uint4 x[2][4];
  read(0, x[0]);
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[u][i] = 0.0f;
#pragma unroll
  for (int n = 0; n < G; ++n) {
    keep_order();
    if (n + 1 < G) read(n + 1, x[(n + 1) & 1]);
    keep_order();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sc[i % NU] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          __builtin_bit_cast(f16x8_t, x[n & 1][i]), q[J * n + i / NU], sc[i % NU], 0, 0, 0);
  }
  keep_order();
}
// O^T += V^T P^T of 64 positions; v: the lane's unit of the first operand, weights(b): of the b-th
// 16 positions.
template <int D, int NJ, class P>
__device__ __forceinline__ void tile_values(const uint4* v, P weights, f32x16_t (&o)[NJ]) {
  const auto read = [&](int b, uint4 (&x)[NJ]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) x[j] = v[2 * b * D + 32 * j];
  };
  uint4 x[2][NJ];
  read(0, x[0]);
  f16x8_t p = weights(0);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    keep_order();
    f16x8_t next = p;
    if (b < 3) {
      read(b + 1, x[(b + 1) & 1]);
      next = weights(b + 1);
    }
    keep_order();
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, x[b & 1][j]), p,
                                                    o[j], 0, 0, 0);
    p = next;
  }
  keep_order();
}

// Joins the partials of a tile of many rows: few parts, so a thread keeps 4 columns of 4 rows and
// goes through the parts in order.
template <int D, int R>
__device__ __forceinline__ void join_tiles(const Kv4AttnArgs& a, const Tile& t, int first, int n,
                                           int tid) {
  constexpr int LR = D / 4, RS = TILE_THREADS / LR, SIZE = R * (D + 2);
  const __amdgpu_buffer_rsrc_t pr = part_rsrc(a.part);
  const int d = 4 * (tid % LR);
  for (int r0 = tid / LR; r0 < t.n_rho; r0 += 4 * RS) {
    float mm[4], ll[4];
    float4 oo[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      mm[u] = -FLT_MAX;
      ll[u] = 0.0f;
      oo[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int k = 0; k < n; ++k) {
      const int at = (first + k) * SIZE;
      float4 v[4];
      float pm[4], pl[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int rr = min(r0 + u * RS, t.n_rho - 1);
        v[u] = ld4_agent(pr, at + rr * D + d);
        pm[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(pr, (at + R * D + rr) * 4, 0, 16));
        pl[u] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(pr, (at + R * D + R + rr) * 4, 0, 16));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float mx = fmaxf(mm[u], pm[u]);
        const float f0 = __builtin_amdgcn_exp2f(mm[u] - mx), f = __builtin_amdgcn_exp2f(pm[u] - mx);
        mm[u] = mx;
        ll[u] = ll[u] * f0 + pl[u] * f;
        oo[u].x = oo[u].x * f0 + v[u].x * f; oo[u].y = oo[u].y * f0 + v[u].y * f;
        oo[u].z = oo[u].z * f0 + v[u].z * f; oo[u].w = oo[u].w * f0 + v[u].w * f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int rr = r0 + u * RS;
      if (rr < t.n_rho) {
        store_out4(a, t, D, rr, d, oo[u], row_inv(ll[u]));
        if (d == 0) store_lse(a, t, rr, mm[u], ll[u]);
      }
    }
  }
}

template <int D, int FMT>
__global__ __launch_bounds__(TILE_THREADS, 2) void kv4_attn_tiles_kernel(Kv4AttnArgs a) {
  constexpr int HV = tile_halves(D), R = tile_rows(D), NU = 2 / HV, N = D / 64, NJ = D / 32 / HV;
  constexpr int NE = TileStage<D>::NE, SIZE = R * (D + 2);
  constexpr int NOWHERE = 0x40000000;  // place of a step that is not there: behind every row
  __shared__ uint4 lds_k[2][k_unit(D, D / 8)];
  __shared__ uint4 lds_v[2][TILE_POS / 8][D];
  __shared__ uint32_t lds_bad[4][8];  // positions of each block whose V scale is not usable
  __shared__ uint4 lds_p[HV == 2 ? 4 : 1][HV == 2 ? 4 : 1][64];
  __shared__ float lds_m[HV == 2 ? 4 : 1][2][32];
  __shared__ int lds_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = wave >> 2;
  // the wavefront's 32 rows, and (D = 256) its half of the positions and columns
  const int rows32 = HV == 2 ? 2 * group + ((wave & 3) >> 1) : wave, half = HV == 2 ? wave & 1 : 0;
  const int q32 = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % a.w.Hkv;
  Piece f;
  if (!find_piece(a, R, blockIdx.x / a.w.Hkv, f)) return;
  const Layout<D> L(a.w);
  const TileMap<D> map(tid);
  const TileOffsets<D> off(a.w, L, map);
  // row m of an A operand of K -> its position within 32
  const int k_tok = 16 * (q32 >> 4) + 8 * ((q32 >> 2) & 1) + 4 * ((q32 >> 3) & 1) + (q32 & 3);
  // the sign of the scale goes to Q; 1e-30 stands for a scale of 0 (equal weights all the same)
  const float c = fmaxf(fabsf(a.scale * LOG2E), 1e-30f), move_by = MOVE / c;
  Tile t;
  tile_of(a, f.s, f.b, f.tile, head, R, t);
  const int s0 = f.s0;
  const bool whole = f.n == 1;
  if (t.s.len > t.s.cap && s0 == 0 && tid == 0) report(a.w.status, ST_LENGTH);
  const int last = min(f.s1, t.n_steps), n_turns = last > s0 ? (last - s0 + 1) >> 1 : 0;
  const int my0 = 32 * rows32;  // first of the wavefront's rows
  const bool busy = my0 < t.n_rho;
  // positions of the wavefront's first and last row
  const int p_first = t.s.len - t.s.n;
  const int w_lo = p_first + row_of(a, t.rho0 + min(my0, t.n_rho - 1));
  const int w_hi = p_first + row_of(a, t.rho0 + min(my0 + 31, t.n_rho - 1));
  const auto edge_at = [&](int t0, int lo, int hi) {
    return t0 + KV4_STEP - 1 > lo ||
           (a.window > 0 && t0 <= hi - a.window && t0 + KV4_STEP > a.sinks);
  };
  // 64 steps from list0 on, one a lane: position, offset of the codes in the cache, how far the
  // scales are from there; and which steps some row of the workgroup, or of the wavefront,
  // does not see whole.  A step that is not there is read somewhere and seen nowhere.
  int list0 = s0, l_pos = NOWHERE, l_scales = 0;
  int64_t l_codes = 0;
  uint64_t edges = 0, my_edges = 0;
  const auto load_list = [&](int from) {
    list0 = from;
    const int at = position_of(t, min(from + lane, last - 1));
    int page = a.w.table[(int64_t)t.b * a.w.max_pages + (at >> a.w.page_shift)];
    const bool there = page >= 0 && page < a.w.num_pages, mine = from + lane < last;
    if (!there && mine) report(a.w.status, ST_PAGE);
    page = there ? page : 0;
    l_pos = there && mine ? at : NOWHERE;
    const int in_page = at & ((1 << a.w.page_shift) - 1);
    l_codes = page * a.w.page_bytes + (int64_t)head * a.w.head_bytes + in_page * (D / 2);
    l_scales = ((in_page << L.n_shift) << 1) - in_page * (D / 2);
    edges = __ballot(edge_at(l_pos, t.p_lo, t.p_hi));
    my_edges = __ballot(edge_at(l_pos, w_lo, w_hi));
  };
  // where the thread reads its codes of a turn
  const uint8_t* codes = a.w.cache;
  uint32_t scales = 0;
  const auto go_to = [&](int turn) {
    const int i = s0 + 2 * turn + group - list0;
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(l_codes >> 32), i);
    codes = a.w.cache + (int64_t)((uint64_t)hi << 32 |
                                  (uint32_t)__builtin_amdgcn_readlane((int)l_codes, i));
    scales = (uint32_t)__builtin_amdgcn_readlane(l_scales, i);
  };
  TileStage<D> st;
  uint32_t vs_now[NE][4];  // V scales of the turn whose V is decoded next
  const auto decode_k = [&](int turn) {  // K of a turn, and its V scales to vs_now
    const _Float16 s1 = (_Float16)bf16_to_f32(st.ks);
    const f16x2_t s = {s1, s1}, s24 = s * (f16x2_t){(_Float16)-24.0f, (_Float16)-24.0f};
    const f16x2_t s4[4] = {s, s, s, s}, z4[4] = {s24, s24, s24, s24};
#pragma unroll
    for (int i = 0; i < N; ++i)
      lds_k[turn & 1][k_unit(D, map.kd + i) + map.tok] =
          __builtin_bit_cast(uint4, decode_f16<FMT>(st.k[i], s4, z4));
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      vs_now[e][0] = st.vs[e].x; vs_now[e][1] = st.vs[e].y;
      vs_now[e][2] = st.vs[e].z; vs_now[e][3] = st.vs[e].w;
    }
    if ((edges >> (s0 + 2 * turn + group - list0)) & 1) {
      // scales that fp16 cannot take: cleared, and the rows that see them are told.  (In a step
      // that all rows see whole they do their damage by themselves.)
      uint32_t over[4], any_over = 0, any = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        over[i] = above_limit<FMT>(vs_now[0][i]);
#pragma unroll
        for (int e = 1; e < NE; ++e) over[i] |= above_limit<FMT>(vs_now[e][i]);
        any_over |= over[i];
      }
      if (__ballot(any_over != 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t h16 = (i & 1) ? 0xFFFF0000u : 0x0000FFFFu;
          const bool bad = (over[i / 2] & h16) != 0;
          any |= __ballot(bad) ? 1u << i : 0u;
#pragma unroll
          for (int e = 0; e < NE; ++e) vs_now[e][i / 2] &= bad ? ~h16 : ~0u;
        }
      }
      if (lane == 0) lds_bad[turn & 3][wave] = any;
    }
  };
  const auto decode_v = [&](int turn) {
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      f16x2_t vs[4], vs24[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int i0 = value_at<FMT>(2 * i), i1 = value_at<FMT>(2 * i + 1);
        vs[i] = f16x2_t{
            (_Float16)((i0 & 1) ? bf16_hi(vs_now[e][i0 / 2]) : bf16_lo(vs_now[e][i0 / 2])),
            (_Float16)((i1 & 1) ? bf16_hi(vs_now[e][i1 / 2]) : bf16_lo(vs_now[e][i1 / 2]))};
        vs24[i] = vs[i] * (f16x2_t){(_Float16)-24.0f, (_Float16)-24.0f};
      }
#pragma unroll
      for (int i = 2 * e; i < N && i < 2 * e + 2; ++i)
        lds_v[turn & 1][map.blk][map.vd + v_step(i)] =
            __builtin_bit_cast(uint4, decode_f16<FMT>(st.v[i], vs, vs24));
    }
  };

  if (n_turns > 0) {
    load_list(s0);
    go_to(0);
    tile_load_k<D>(codes, scales, off, st);
  }
  f16x8_t q[D / 16];
  int pos;
  {
    const int rho = t.rho0 + my0 + q32;
    const bool on = my0 + q32 < t.n_rho;
    const int i = row_of(a, rho), hh = t.head * a.r + rho - i * a.r;
    pos = on ? p_first + i : -1;
    const uint16_t* p = a.q + (int64_t)(t.s.row0 + i) * a.q_stride + (int64_t)hh * D + 8 * h;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (on) u = *reinterpret_cast<const uint4*>(p + 16 * j);
      const uint32_t uw[4] = {u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = value_at<FMT>(e);
        q[j][e] = (_Float16)((d & 1) ? bf16_hi(uw[d / 2]) : bf16_lo(uw[d / 2]));
      }
    }
  }
  f32x16_t o[NJ], sc[NU];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
  float m = -FLT_MAX, l = 0.0f;  // m: of the scores before scaling
  // hides what the rows do not see of a turn's scores; the lane's largest score
  const auto mask_scores = [&](int turn) {
    const int i0 = s0 + 2 * turn + (HV == 2 ? half : 0) - list0;
    constexpr uint64_t UM = (1u << NU) - 1;
    if ((edges >> i0) & UM) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        uint32_t bad = 0;
        if ((edges >> (i0 + u)) & 1)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            bad |= lds_bad[turn & 3][4 * (HV == 2 ? half : u) + b] << (8 * b);
        if (!((my_edges >> (i0 + u)) & 1) && bad == 0) continue;
        const int t0 = __builtin_amdgcn_readlane(l_pos, i0 + u);
        // against the constant offset of a register's position
        const int to = pos - t0 - 8 * h, from = a.window > 0 ? max(to, -1) - a.window : -1000;
        const int first = a.sinks - t0 - 8 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = 16 * (i >> 3) + (i & 7);
          const bool seen = at <= to && (at > from || at < first);
          sc[u][i] = seen ? sc[u][i] : -INFINITY;
        }
        if (bad) {
          const uint32_t mine = bad >> (8 * h);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((mine >> (16 * (i >> 3) + (i & 7))) & 1 && sc[u][i] != -INFINITY)
              sc[u][i] = NAN;
        }
      }
    }
    float mx = fmaxf(sc[0][0], sc[NU - 1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = fmaxf(fmaxf(mx, sc[0][i]), sc[NU - 1][i]);
    return mx;
  };
  const auto move_reference = [&](float mx) {  // mx: of the row
    if (__ballot(mx > m + move_by)) {
      if constexpr (HV == 1) mx = fmaxf(mx, __shfl_xor(mx, 32));
      mx = fmaxf(mx, m);
      const float f = __builtin_amdgcn_exp2f((m - mx) * c);
      m = mx;
      l *= f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[j] *= f;
    }
    return P_SHIFT - fmaxf(m * c, -FLT_MAX);
  };
  // the weights of the b-th 16 positions of the wavefront
  const auto weights = [&](int b, float ref) {
    float e[8];
    f16x8_t w;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e[i] = __builtin_amdgcn_exp2f(fmaf(sc[b >> 1][8 * (b & 1) + i], c, ref));
    l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (_Float16)e[value_at<FMT>(i)];
    return w;
  };
  if constexpr (HV == 1) {
    if (n_turns > 0) {
      const auto decode_next = [&](int k) {
        if (k >= n_turns) return;
        decode_k(k);
        decode_v(k);
        if (k + 1 >= n_turns) return;
        // (the list has the scores of turn k - 1 and K of turn k + 1)
        if (s0 + 2 * k + 4 > list0 + 64) load_list(s0 + 2 * (k - 1));
        go_to(k + 1);
        tile_load_k<D>(codes, scales, off, st);
        tile_load_v<D>(codes, off, st);
      };
      tile_load_v<D>(codes, off, st);
      decode_next(0);
      __syncthreads();
#pragma unroll 1
      for (int turn = 0; turn < n_turns; ++turn) {
        __builtin_amdgcn_s_setprio(1);
        if (group == 1) decode_next(turn + 1);
        __builtin_amdgcn_s_setprio(0);
        tile_scores<D, NU>(&lds_k[turn & 1][k_unit(D, h) + k_tok], q, sc);
        const float ref = move_reference(mask_scores(turn));
        __builtin_amdgcn_s_setprio(1);
        tile_values<D, NJ>(&lds_v[turn & 1][h][q32], [&](int b) { return weights(b, ref); }, o);
        __builtin_amdgcn_s_setprio(0);
        if (group == 0) decode_next(turn + 1);
        __syncthreads();
      }
    }
  } else if (n_turns > 0) {
    // K of turn k and V of the turn before from their codes to LDS, and the next codes' loads
    const auto decode_turn = [&](int k) {
      if (k > n_turns) return;
      decode_v(k - 1);
      if (k >= n_turns) return;
      decode_k(k);
      tile_load_v<D>(codes, off, st);
      if (k + 1 >= n_turns) return;
      // (the list has the scores of turn k - 2 at the earliest, K of turn k + 1 at the latest)
      if (s0 + 2 * k + 4 > list0 + 64) load_list(s0 + 2 * max(k - 2, 0));
      go_to(k + 1);
      tile_load_k<D>(codes, scales, off, st);
    };
    const auto values = [&](int turn) {
      tile_values<D, NJ>(&lds_v[turn & 1][h][32 * NJ * half + q32], [&](int b) {
        return __builtin_bit_cast(f16x8_t, lds_p[rows32][b][lane]);
      }, o);
    };
    decode_k(0);
    tile_load_v<D>(codes, off, st);
    if (n_turns > 1) {
      go_to(1);
      tile_load_k<D>(codes, scales, off, st);
    }
    __syncthreads();
    if (group == 1) {  // half a turn behind group 0
      decode_turn(1);
      __syncthreads();
    }
#pragma unroll 1
    for (int turn = 0; turn < n_turns; ++turn) {
      // phase M
      __builtin_amdgcn_s_setprio(1);
      if (turn > 0) values(turn - 1);
      tile_scores<D, NU>(&lds_k[turn & 1][k_unit(D, h) + 32 * half + k_tok], q, sc);
      __builtin_amdgcn_s_setprio(0);
      float mx = mask_scores(turn);
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      if (h == 0) lds_m[rows32][half][q32] = mx;
      __syncthreads();
      // phase A
      mx = fmaxf(mx, lds_m[rows32][half ^ 1][q32]);
      const float ref = move_reference(mx);
#pragma unroll
      for (int b = 0; b < 2 * NU; ++b)
        lds_p[rows32][2 * half + b][lane] = __builtin_bit_cast(uint4, weights(b, ref));
      decode_turn(turn + 1 + group);
      __syncthreads();
    }
    values(n_turns - 1);
    if (group == 0) __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if constexpr (HV == 2) {
    if (h == 0) lds_m[rows32][half][q32] = l;
    __syncthreads();
    l = lds_m[rows32][0][q32] + lds_m[rows32][1][q32];
  }
  const float m2 = l != 0.0f ? m * c : -FLT_MAX;  // in powers of 2, as the other kernel's
  const int row = my0 + q32, partial = head * 2 * a.n_parts + f.partial;
  const int d0 = 32 * NJ * half + 4 * h;
  if (row < t.n_rho) {
    if (whole) {
      const float inv = row_inv(l);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          store_out4(a, t, D, row, d0 + 32 * j + 2 * i,
                     make_float4(o[j][i], o[j][i + 1], o[j][i + 2], o[j][i + 3]), inv);
      if (d0 == 0) store_lse(a, t, row, m2, l);
    } else {
      const __amdgpu_buffer_rsrc_t pr = part_rsrc(a.part);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          st4_agent(pr, partial * SIZE + row * D + d0 + 32 * j + 2 * i,
                    make_float4(o[j][i], o[j][i + 1], o[j][i + 2], o[j][i + 3]));
      if (d0 == 0) {
        st_sc1(a.part, (size_t)partial * SIZE + R * D + row, m2);
        st_sc1(a.part, (size_t)partial * SIZE + R * D + R + row, l);
      }
    }
  }
  if (!whole) {
    unsigned* counter = a.counters + head * 2 * a.n_parts + (f.partial - f.index);
    if (last_arriver(counter, (unsigned)f.n, &lds_flag)) {
      join_tiles<D, R>(a, t, partial - f.index, f.n, tid);
      if (tid == 0) st_cnt(counter, 0u);
    }
  }
}

template <int D, int FMT>
hipError_t launch_rows(const Kv4RowsArgs& a, hipStream_t st) {
  const int64_t units = 2 * (int64_t)a.w.Hkv * ((a.w.T >> 3) + 2 * (int64_t)a.w.B);
  const dim3 grid((unsigned)((units + 3) / 4));
  if (a.k)
    kv4_write_kernel<D, FMT><<<grid, 256, 0, st>>>(a, (int)units);
  else
    kv4_read_kernel<D, FMT><<<grid, 256, 0, st>>>(a, (int)units);
  return hipGetLastError();
}

template <int D, int FMT>
hipError_t launch_attn(const Kv4AttnArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)a.w.Hkv * a.n_groups;
  if (a.plan) {
    kv4_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(a, 16 * a.nt);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.nt == kv4_tile_nt(D)) {
    kv4_attn_tiles_kernel<D, FMT><<<grid, TILE_THREADS, 0, st>>>(a);
    return hipGetLastError();
  }
  const auto rows = [&](auto kernel) { kernel<<<grid, 64 * a.waves, 0, st>>>(a); };
  if constexpr (D <= 128) {
    if (a.nt == 2) {
      rows(a.waves == 4 ? kv4_attn_rows_kernel<D, FMT, 2, 4> : kv4_attn_rows_kernel<D, FMT, 2, 8>);
      return hipGetLastError();
    }
  }
  rows(a.waves == 4 ? kv4_attn_rows_kernel<D, FMT, 1, 4> : kv4_attn_rows_kernel<D, FMT, 1, 8>);
  return hipGetLastError();
}
template <template <int, int> class L, class A>
hipError_t by_type(const A& a, int D, int fmt, hipStream_t st) {
  if (fmt == FMT_INT4)
    return D == 64 ? L<64, FMT_INT4>::go(a, st)
                   : D == 128 ? L<128, FMT_INT4>::go(a, st) : L<256, FMT_INT4>::go(a, st);
  return D == 64 ? L<64, FMT_FP4>::go(a, st)
                 : D == 128 ? L<128, FMT_FP4>::go(a, st) : L<256, FMT_FP4>::go(a, st);
}
template <int D, int FMT>
struct Rows {
  static hipError_t go(const Kv4RowsArgs& a, hipStream_t st) { return launch_rows<D, FMT>(a, st); }
};
template <int D, int FMT>
struct Attn {
  static hipError_t go(const Kv4AttnArgs& a, hipStream_t st) { return launch_attn<D, FMT>(a, st); }
};

}  // namespace

hipError_t launch_kv4_write(const Kv4RowsArgs& a, int D, int fmt, hipStream_t st) {
  return by_type<Rows>(a, D, fmt, st);
}
hipError_t launch_kv4_read(const Kv4RowsArgs& a, int D, int fmt, hipStream_t st) {
  return by_type<Rows>(a, D, fmt, st);
}
hipError_t launch_kv4_attention(const Kv4AttnArgs& a, int D, int fmt, hipStream_t st) {
  return by_type<Attn>(a, D, fmt, st);
}

}  // namespace dqg
