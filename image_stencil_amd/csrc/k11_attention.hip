// k11_attention.hip -- cross attention on the matrix cores.
//
//   out = softmax(scale q k^T) v, one pass over the keys with a running maximum
//   and sum: with s = q . k, c = |scale| log2(e) (the sign goes into q) and M the
//   running maximum of c s,  p = 2^(c s - M),  l = sum p,  O = sum p v,  out = O / l.
//
// Both products run as v_mfma_f32_32x32x16 with the queries as columns:
//   S^T (keys x queries) = K Q^T      A = K rows (LDS), B = Q (registers)
//   O^T (d x queries)    = V^T P^T    A = V columns (transposing LDS reads), B = P
// The accumulator of S^T puts keys 8 a + 4 h + (0..3) of a query's 32 into lane
// half h (a = 0..3). The order of a product's inner index is free, so P goes
// from these registers into the second product as it lies, and V's columns are
// read in the same order of keys: P never crosses lanes or LDS. M, l and the
// factor of a rescale belong to a query, which is a lane.
//
// A workgroup of NW waves either shares key tiles of 64 keys, 32 QB query rows
// per wave (SHARED: many queries; RESIDENT: all keys stay in LDS for several row
// tiles), or lets every wave walk key tiles of 32 of its own for the same 32 rows
// and joins the waves' results at the end (few queries, where the read of k and v
// is all the work). K and V arrive by LDS DMA in two or four buffers each, without
// passing registers. A step computes the scores of tile j + 1 beside the
// exponentials of tile j (matrix cores beside vector unit), then adds tile j's p v
// beside the maximum of tile j + 1, and issues the loads of the tiles after. M
// moves only when a row's maximum outgrows it by 2^8, so that most steps scale
// nothing; p stays under 2^8, and its sum in 32 bits.
//
// Rows of k and v that may not be seen are never fetched (an out-of-range
// offset makes the DMA write zeros); their scores start from -infinity, in the
// accumulator (MASK) or after the product (the last tile's end).
//
// What bounds it, measured on MI355Xs: heads of 128, 16384 x 16384 tokens, 16 query
// and 4 key heads, bf16: 1868 to 1977 us on different cards, 1.11 to 1.18 PFLOP/s, the
// rate of a large library product, at the clock the power limit leaves. Heads of
// 64, 3600 x 3600, 16 heads, fp16: 74 to 78 us, 0.68 to 0.72 PFLOP/s: per 32 x 32 scores
// the vector unit is active for about 430 cycles (91 instructions: 16 exponentials
// of 8 cycles each, multiply-adds, sums, conversions and maxima) and the matrix cores
// for 256, and the two hardly overlap (48% and 28% of the time). One token over
// 4 x 32771 keys, 2 heads of 128: 30.9 us, 4.3 TB/s of k and v with the join.
#include <float.h>
#include <math.h>

#include "attention.hpp"
#include "common.hpp"
#include "divide.hpp"
#include "join.hpp"

namespace is {
namespace {

constexpr unsigned kOob = 0xFFFFFFF0u;
constexpr float kLazy = 8.f;   // log2 of how far a row's maximum may outgrow M

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));

struct Args {
  const void *q, *k, *v;
  const uint8_t *mask;
  const int32_t *lengths;
  void *out;
  float *lse;
  float *part;            // splits > 1: O / l of every block, [block][tile row][d]
  float *part_lse;        // and M + log2 l, [block][tile row]
  int64_t qs[3], ks[3], vs[3], os[3], mask_bs;
  int lq, lk, hq, hkv, d, group, rows, row_tiles, splits, split_keys, groups, runs;
  int run;                // row tiles a workgroup goes through
  Divisor by_group, by_runs, by_splits, by_hkv;
  unsigned flip;          // sign bits of a negative scale
  float c;                // |scale| log2(e)
};

// Row pitch of an LDS tile, in 16-byte chunks: a power of two.
constexpr int chunk_pitch(int dp) { return dp <= 32 ? 4 : dp <= 64 ? 8 : dp <= 128 ? 16 : 32; }

// Chunk c of row r lies in slot c ^ f(r) of its row. K is read one chunk of 16
// consecutive rows per pass, V as 4 consecutive rows x 64 bytes: with these f
// both fall on different banks.
template <int CP>
__device__ __forceinline__ int fk(int r) {
  return CP >= 16 ? r & 15 : CP == 8 ? (r >> 1) & 7 : (r >> 2) & 3;
}
template <int CP>
__device__ __forceinline__ int fv(int r) {
  return CP >= 16 ? (r & 3) << 2 : CP == 8 ? (r & 2) << 1 : 0;
}

__device__ __forceinline__ floatx16 mma(_Float16 __attribute__((ext_vector_type(8))) a,
                                        _Float16 __attribute__((ext_vector_type(8))) b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mma(__bf16 __attribute__((ext_vector_type(8))) a,
                                        __bf16 __attribute__((ext_vector_type(8))) b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// N operations of 16 bytes per lane from a buffer straight into LDS, operation i
// to dst + i * STEP + 16 lane (zeros for an offset outside the buffer). Written as
// instructions because the compiler takes the builtin for a store that any later
// transposing LDS read may meet, and waits for it there; the kernel's own waits
// (arrived) are what is needed. They have no output register, so nothing is open
// while they run. The s_nop 4 keeps a descriptor that a vector instruction brought
// to scalar registers (a spill) five wait states from its first use.
#define IS_DMA16(O) "buffer_load_dwordx4 " O ", %1, 0 offen lds\n\t"
#define IS_NEXT "s_add_u32 m0, m0, %c2\n\ts_nop 0\n\t"
template <int N, int STEP>
__device__ __forceinline__ void dma16(uintx4 rs, unsigned dst, const unsigned *o) {
  if constexpr (N >= 4) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\t" IS_DMA16("%3") IS_NEXT IS_DMA16("%4") IS_NEXT IS_DMA16("%5")
                         IS_NEXT IS_DMA16("%6")
                     :
                     : "s"(dst), "s"(rs), "n"(STEP), "v"(o[0]), "v"(o[1]), "v"(o[2]), "v"(o[3])
                     : "memory", "scc");
    if constexpr (N > 4) dma16<N - 4, STEP>(rs, dst + 4 * STEP, o + 4);
  } else if constexpr (N == 2) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\t" IS_DMA16("%3") IS_NEXT IS_DMA16("%4")
                     :
                     : "s"(dst), "s"(rs), "n"(STEP), "v"(o[0]), "v"(o[1])
                     : "memory", "scc");
  } else {
    static_assert(N == 1, "a power of two");
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\t" IS_DMA16("%2")
                     :
                     : "s"(dst), "s"(rs), "v"(o[0])
                     : "memory");
  }
}
#undef IS_DMA16
#undef IS_NEXT
// One operation of 4 bytes per lane.
__device__ __forceinline__ void dma4(uintx4 rs, unsigned dst, unsigned off) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                   :
                   : "s"(dst), "v"(off), "s"(rs)
                   : "memory");
}
// A buffer descriptor for them.
__device__ __forceinline__ uintx4 descriptor(uint64_t at, unsigned bytes) {
  return uintx4{(unsigned)at, (unsigned)(at >> 32) & 0xffffu, bytes, (unsigned)kBufferFlags};
}

// s_waitcnt operand: at most n vector-memory operations outstanding.
constexpr int wait_vm(int n) { return 0x0F70 | (n & 15) | (n >> 4) << 14; }

// The value of the lane 32 away, joined by max or sum.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The value is computed before this point (the compiler would move sums to where
// they are used, behind the products they should run beside).
__device__ __forceinline__ void pin(float &x) { __asm__ volatile("" : "+v"(x)); }

constexpr bool in_time(int f_k, int mb, int operands, int lag, int pairs, int last) {
  for (int f = 0; f < operands; ++f)
    if ((f_k + f * mb - 2 * lag) * pairs / last < 4 * (f + 1)) return false;
  return true;
}

template <int DP, int NW, bool SHARED, bool MASK>
struct Geo {
  static constexpr int CP = chunk_pitch(DP);
  static constexpr int KT = SHARED ? 64 : 32;              // keys of a tile
  static constexpr int NKB = KT / 32;
  static constexpr int TILE = KT * CP * 16;                // bytes of a K or V tile
  static constexpr int LOADERS = SHARED ? NW : 1;          // waves that bring a tile
  static constexpr int NI = KT * CP / 64 / LOADERS;        // 1 KB DMA operations of a wave and tile
  // Buffers of K (as many of V), and steps between the barriers of shared tiles.
  static constexpr int RB = SHARED && CP <= 8 ? 4 : 2, SP = RB / 2;
  static constexpr int RING = 2 * RB * TILE;
  static constexpr int JOIN_PITCH = DP + 4;                // floats
  static constexpr int RINGS = SHARED ? RING : NW * RING;
  static constexpr int JOIN = SHARED ? 0 : NW * 32 * (JOIN_PITCH + 2) * 4;
  static constexpr int MASKS = RINGS > JOIN ? RINGS : JOIN;   // a wave's mask bytes, then its bias
  static constexpr int MASK_SLOT = 256, MASK_SLOTS = 4;
  static constexpr int MASK_WAVE = MASK_SLOTS * MASK_SLOT + 2 * KT * 4;
  static constexpr int BYTES = MASKS + (MASK ? NW * MASK_WAVE : 0);
  static constexpr int WAVES = BYTES <= 80 * 1024 && NW == 4 ? 2 : 1;   // per SIMD: two workgroups in a CU's LDS
  static_assert(NI >= 1 && NI * 64 * LOADERS == KT * CP, "whole DMA operations");
};

// RESIDENT (with SHARED): all keys fit the buffers, and a workgroup goes through
// a.run row tiles with them, the next one's queries on their way.
template <typename T, int DP, int QB, int NW, bool SHARED, bool RESIDENT, bool MASK>
__global__ __launch_bounds__(NW * 64, (Geo<DP, NW, SHARED, MASK>::WAVES)) void is_k11_attention(const Args a) {
  typedef T T8 __attribute__((ext_vector_type(8)));
  typedef T T2 __attribute__((ext_vector_type(2)));
  typedef float F2 __attribute__((ext_vector_type(2)));
  typedef short S4 __attribute__((ext_vector_type(4)));
  using G = Geo<DP, NW, SHARED, MASK>;
  constexpr int CP = G::CP, KT = G::KT, NKB = G::NKB, NI = G::NI, KK = DP / 16, MB = DP / 32, RB = G::RB;
  constexpr int ROWS = SHARED ? 32 * QB * NW : 32;
  __shared__ __attribute__((aligned(1024))) char lds[G::BYTES];
  lds_poison(lds, sizeof(lds));

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n32 = lane & 31, half = lane >> 5;

  // Workgroup -> (entry and key head, split, row tile). Row tiles of a group
  // read the same keys, so a group stays on one XCD: groups are dealt to the 8
  // XCDs in turn, or in one run of consecutive tiles where 8 does not divide them.
  const bool dealt = (a.groups & 7) == 0;
  const int place = dealt ? (int)(blockIdx.x >> 3) : xcd_remap(blockIdx.x, gridDim.x);
  const int turn = divide(place, a.by_runs);
  const int g = dealt ? turn * 8 + (int)(blockIdx.x & 7) : turn;
  const int rt0 = (place - turn * a.runs) * (RESIDENT ? a.run : 1);
  const int bh = divide(g, a.by_splits), split = g - bh * a.splits;
  const int b = divide(bh, a.by_hkv), hk = bh - b * a.hkv;

  int len = a.lk;
  if (a.lengths) len = min(len, max(0, a.lengths[b]));
  const int first = split * a.split_keys;
  const int keys = max(0, min(len - first, a.split_keys));
  const int tiles = (keys + KT - 1) / KT;
  // Tiles of this wave, and the first key of its j-th.
  const int nt = SHARED ? tiles : (tiles - wave + NW - 1) / NW;
  auto tile_key = [&](int j) { return (SHARED ? j : j * NW + wave) * KT; };

  // ---- DMA: operation i of a wave brings slots 64 (i LOADERS + wave) + lane.
  const int ktok = (int)(a.ks[1] * 2), vtok = (int)(a.vs[1] * 2);   // bytes, at most 2^24
  const char *kbase = static_cast<const char *>(a.k) + (b * a.ks[0] + hk * a.ks[2] + first * a.ks[1]) * 2;
  const char *vbase = static_cast<const char *>(a.v) + (b * a.vs[0] + hk * a.vs[2] + first * a.vs[1]) * 2;
  char *ring = lds + (SHARED ? 0 : wave * G::RING);
  const unsigned lds_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
  const unsigned ring_at = lds_at + (unsigned)(SHARED ? 0 : wave * G::RING);
  int drow[NI];
  unsigned koff[NI], voff[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = (i * G::LOADERS + (SHARED ? wave : 0)) * 64 + lane;
    const int r = slot / CP, kc = slot % CP ^ fk<CP>(r), vc = slot % CP ^ fv<CP>(r);
    drow[i] = r;
    koff[i] = kc * 8 < a.d ? (unsigned)(r * ktok + kc * 16) : kOob;
    voff[i] = vc * 8 < a.d ? (unsigned)(r * vtok + vc * 16) : kOob;
  }
  // The next K or V tile into LDS at dst: its rows that may be seen; a tile past
  // the keys gets zeros. The descriptor spans a whole tile: rows that may not be
  // read have an offset outside it.
  uint64_t knext = (uint64_t)(uintptr_t)kbase + (uint64_t)((int64_t)tile_key(0) * ktok);
  uint64_t vnext = (uint64_t)(uintptr_t)vbase + (uint64_t)((int64_t)tile_key(0) * vtok);
  const int stride = SHARED ? KT : NW * KT;   // keys from one of this wave's tiles to the next
  const uint64_t kstep = (uint64_t)((int64_t)stride * ktok), vstep = (uint64_t)((int64_t)stride * vtok);
  const unsigned kspan = (unsigned)((KT - 1) * ktok + a.d * 2), vspan = (unsigned)((KT - 1) * vtok + a.d * 2);
  auto issue = [&](uint64_t &at, uint64_t step, unsigned span, const unsigned *off, int left, unsigned dst,
                   uint64_t bits) {
    const uintx4 rs = descriptor(at, span);
    at += step;
    unsigned o[NI];
    if constexpr (MASK) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        // All ones where the row's bit is set: one bit-field extract and one select.
        constexpr int SPAN = G::LOADERS * 64 / CP;   // rows of an operation
        const int r = drow[i];
        const bool low = KT == 32 || (SPAN <= 32 ? i * SPAN < 32 : r < 32);
        const int word = low ? (int)bits : (int)(bits >> 32);
        const unsigned m = (unsigned)__builtin_amdgcn_sbfe(word, (unsigned)(r & 31), 1);
        o[i] = (off[i] & m) | (kOob & ~m);
      }
    } else if (left < KT) {
#pragma unroll
      for (int i = 0; i < NI; ++i) o[i] = drow[i] < left ? off[i] : kOob;
      dma16<NI, G::LOADERS * 1024>(rs, dst + (SHARED ? wave : 0) * 1024u, o);
      return;
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) o[i] = off[i];
    }
    dma16<NI, G::LOADERS * 1024>(rs, dst + (SHARED ? wave : 0) * 1024u, o);
  };
  auto issue_k = [&](int j, int buffer, uint64_t bits) {   // tiles in order
    issue(knext, kstep, kspan, koff, keys - tile_key(j), ring_at + buffer * G::TILE, bits);
  };
  auto issue_v = [&](int j, int buffer, uint64_t bits) {
    issue(vnext, vstep, vspan, voff, keys - tile_key(j), ring_at + (RB + buffer) * G::TILE, bits);
  };
  // At most N of this wave's DMA operations still out, then (a shared tile)
  // every wave's.
  auto arrived = [&](auto n) {
    constexpr int N = decltype(n)::value;
    static_assert(N < 64, "vmcnt");
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm(N));
    if constexpr (SHARED) __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
  };
  // Mask bytes: the words from tile j's first on, into slot j % 4 (tiles in order).
  // The descriptor ends with the word of the last key; a first word may begin with
  // up to three bytes before it.
  const unsigned masks_at = lds_at + (unsigned)(G::MASKS + wave * G::MASK_WAVE);
  const uint64_t mask0 = MASK ? (uint64_t)(uintptr_t)a.mask + (uint64_t)(b * a.mask_bs + first) : 0;
  const int skip = (int)(mask0 & 3);
  const uintx4 mask_rs = descriptor(mask0 & ~(uint64_t)3, (unsigned)((keys + skip + 3) & ~3));
  unsigned mask_off = (unsigned)(tile_key(0) + lane * 4);
  auto issue_mask = [&](int j) {
    if constexpr (MASK) {
      dma4(mask_rs, masks_at + (unsigned)(j & (G::MASK_SLOTS - 1)) * G::MASK_SLOT, mask_off);
      mask_off += (unsigned)stride;
    }
  };
  // A bit for every key of tile j that may be seen; its two parts, the read of a
  // byte per lane and the vote, may stand apart.
  auto mask_byte = [&](int j) -> uint8_t {
    if constexpr (!MASK) return 0;
    return (uint8_t)lds[G::MASKS + wave * G::MASK_WAVE + (j & (G::MASK_SLOTS - 1)) * G::MASK_SLOT + skip + lane % KT];
  };
  uint64_t visible = 0;   // of all tiles so far
  auto vote = [&](int j, uint8_t byte) -> uint64_t {
    if constexpr (!MASK) return 0;
    const uint64_t bits = __ballot(lane < KT && tile_key(j) + lane < keys && byte != 0);
    visible |= bits;
    return bits;
  };
  auto seen = [&](int j) -> uint64_t { return vote(j, mask_byte(j)); };

  // ---- Queries: B operands, lane = row n32, elements 16 kk + 8 half .. + 7.
  T8 qf[QB][KK];
  uintx4 qw[QB][KK];   // of the row tile after, on their way
  auto load_q = [&](int rt) {
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      const int r = rt * ROWS + (SHARED ? wave * 32 * QB : 0) + qb * 32 + n32;
      const int i = divide(r, a.by_group), h = hk * a.group + r - i * a.group;
      const T *p = static_cast<const T *>(a.q) + b * a.qs[0] + i * a.qs[1] + h * a.qs[2];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        qw[qb][kk] = uintx4{0, 0, 0, 0};
        if (r < a.rows && (2 * kk + half) * 8 < a.d)
          qw[qb][kk] = *reinterpret_cast<const uintx4 *>(p + (2 * kk + half) * 8);
      }
    }
  };
  auto take_q = [&]() {
#pragma unroll
    for (int qb = 0; qb < QB; ++qb)
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) qf[qb][kk] = __builtin_bit_cast(T8, qw[qb][kk] ^ a.flip);
  };
  load_q(rt0);

  // ---- LDS read addresses (bytes in a tile).
  const int kaddr = n32 * CP * 16 + ((half ^ fk<CP>(n32)) * 16);          // ^ 32 kk
  const int i16 = lane & 15, vr = 4 * half + (i16 >> 2);
  const int vaddr = vr * CP * 16 + (((2 * ((lane >> 4) & 1) + ((i16 >> 1) & 1)) ^ fv<CP>(vr)) * 16) + (i16 & 1) * 8;  // ^ 64 mb
  float *bias = reinterpret_cast<float *>(lds + G::MASKS + wave * G::MASK_WAVE + G::MASK_SLOTS * G::MASK_SLOT);

  typedef floatx16 Scores[QB][NKB];
  floatx16 o[QB][MB];
  float m[QB], l[QB];

  // A operands in the order of their use: F_K of a K tile, F_V of a V tile.
  constexpr int F_K = NKB * KK, F_V = NKB * 2 * MB;
  auto k_operand = [&](int buffer, int f) -> T8 {
    const char *p = ring + buffer * G::TILE + (f / KK) * 32 * CP * 16 + (kaddr ^ (f % KK * 32));
    return *reinterpret_cast<const T8 *>(p);
  };
  auto v_operand = [&](int buffer, int f) -> T8 {
    typedef __attribute__((address_space(3))) S4 *P;
    const char *p = ring + (RB + buffer) * G::TILE + (f / MB) * 16 * CP * 16 + (vaddr ^ (f % MB * 64));
    const S4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
    const S4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 8 * CP * 16));
    return __builtin_bit_cast(T8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // What the scores of 32 keys start from.
  auto start = [&](int slot, int kb) -> floatx16 {
    floatx16 init;
#pragma unroll
    for (int e = 0; e < 16; ++e) init[e] = 0.f;
    if constexpr (MASK) {
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const floatx4 f = *reinterpret_cast<const floatx4 *>(bias + slot * KT + kb * 32 + 2 * e + 4 * half);
#pragma unroll
        for (int u = 0; u < 4; ++u) init[e + u] = f[u];
      }
    }
    return init;
  };
  auto set_bias = [&](int slot, uint64_t bits) {   // of a tile: slot tile % 2
    if constexpr (MASK) {
      if (lane < KT) bias[slot * KT + lane] = __builtin_amdgcn_inverse_ballot_w64(bits) ? 0.f : -INFINITY;
    }
  };
  // The largest score of every row, in M's unit; half of the lanes' maximum
  // (top) comes from the caller.
  auto maximum = [&](const Scores &s, float *top) {
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      float x = s[qb][0][0];
#pragma unroll
      for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e) x = fmaxf(x, s[qb][kb][e]);
      top[qb] = x;
    }
  };
  // The end of the last tile: keys past it leave, and its maximum is taken again.
  auto cut = [&](Scores &s, int j, float *top) {
    if constexpr (!MASK) {
      const int left = keys - tile_key(j);
      if (left >= KT) return;
      int mine = left - 4 * half;
      __asm__ volatile("" : "+v"(mine));   // kept from leaving a loop over row tiles as 32 masks
#pragma unroll
      for (int qb = 0; qb < QB; ++qb)
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            s[qb][kb][e] = kb * 32 + 8 * (e >> 2) + (e & 3) < mine ? s[qb][kb][e] : -INFINITY;
            __builtin_amdgcn_sched_barrier(0);   // one comparison at a time: 32 at once spill
          }
      maximum(s, top);
    }
  };
  // M follows a row's maximum when that outgrows it, and O and l follow M.
  auto follow = [&](const float *lane_top) {
    bool grow = false;
    float top[QB];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      top[qb] = max_halves(lane_top[qb]) * a.c;
      grow |= top[qb] > m[qb] + kLazy;
    }
    if (!__any(grow)) return;
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      const float next = fmaxf(m[qb], top[qb]);
      const float f = __builtin_amdgcn_exp2f(m[qb] - next);
      m[qb] = next;
      l[qb] *= f;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[qb][mb][e] *= f;
    }
  };
  // Two exponentials in three parts, which run in slots of their own so that none
  // waits for the one before it: the exponents, their powers, and p: rounded to T
  // for the second product (the matrix cores take no wider operand), while the sum
  // l takes it in 32 bits.
  auto exponents = [&](float s0, float s1, int qb) -> F2 {
    return F2{__builtin_fmaf(s0, a.c, -m[qb]), __builtin_fmaf(s1, a.c, -m[qb])};
  };
  auto powers = [&](F2 x) -> F2 { return F2{__builtin_amdgcn_exp2f(x[0]), __builtin_amdgcn_exp2f(x[1])}; };
  auto weights = [&](F2 p, float &sum) -> unsigned {
    sum += p[0];
    sum += p[1];
    return __builtin_bit_cast(unsigned, __builtin_convertvector(p, T2));
  };

  // One step: scores of the next tile (NEXT: into n, from the K buffer after B)
  // beside the exponentials of s, then s's p v (V buffer B) beside the next maximum.
  // A slot is one A operand's products and what the vector unit does in their 32
  // cycles each; the fences keep the order, since a wave issues in order and the
  // compiler would put each kind in a run of its own. Operands are read kAhead
  // slots early. v_here() precedes the first read of the V tile; beside(slot) is
  // what a slot carries of the loads to come (the scalar work of a descriptor
  // takes as long as a product).
  auto step = [&](auto buffer, auto next, const Scores &s, Scores &n, float *top, auto v_here, auto beside) {
    const int B = buffer;   // a constant where the loop is unrolled
    constexpr int NEXT = decltype(next)::value;
    constexpr int FIRST = NEXT ? 0 : F_K, SLOTS = F_K + F_V;
    constexpr int kAhead = 3;
    // Pairs of p: part one of pair i in slot i LAST / PAIRS, the others LAG slots
    // later each; the last four must be there at slot F_K + F_V - MB.
    constexpr int PAIRS = NKB * 8, LAG = F_K < 4 ? 0 : 1, LAST = F_K + F_V - MB - 2 * LAG;
    static_assert(in_time(F_K, MB, NKB * 2, LAG, PAIRS, LAST), "an operand of P is whole before its first product");
    T8 op[kAhead + 1];
    auto fetch = [&](auto f) {
      constexpr int F = decltype(f)::value;
      if constexpr (F < F_K) op[F % (kAhead + 1)] = k_operand((B + 1) % RB, F);
      else if constexpr (F < SLOTS) op[F % (kAhead + 1)] = v_operand(B, F - F_K);
    };
    F2 x[QB][PAIRS];
    uintx4 p[QB][NKB * 2];
    float sum[QB][2] = {};
    // Parts of the pairs [from, to).
    auto part = [&](auto which, auto from, auto to) {
      constexpr int W = decltype(which)::value, P0 = decltype(from)::value, P1 = decltype(to)::value;
      static_for<(P1 > P0 ? P1 - P0 : 0)>([&](auto k) {
        constexpr int P = P0 + decltype(k)::value;
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) {
          if constexpr (W == 0) x[qb][P] = exponents(s[qb][P / 8][2 * (P % 8)], s[qb][P / 8][2 * (P % 8) + 1], qb);
          if constexpr (W == 1) x[qb][P] = powers(x[qb][P]);
          if constexpr (W == 2) p[qb][P / 4][P % 4] = weights(x[qb][P], sum[qb][P & 1]);
        }
      });
    };
    constexpr bool EARLY = !NEXT || F_K < kAhead;   // the first operands reach into the V tile
    // What the scores start from is read as early as the operands.
    auto begin = [&](auto block) {
      constexpr int kb = decltype(block)::value;
      const floatx16 init = start((B + 1) % 2, kb);
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) n[qb][kb] = init;
    };
    if constexpr (EARLY) v_here();
    if constexpr (NEXT) begin(std::integral_constant<int, 0>{});
    static_for<kAhead>([&](auto i) { fetch(std::integral_constant<int, FIRST + decltype(i)::value>{}); });
    if constexpr (!NEXT)
      static_for<3>([&](auto w) { part(w, std::integral_constant<int, 0>{}, std::integral_constant<int, PAIRS>{}); });
    static_for<SLOTS - FIRST>([&](auto i) {
      constexpr int U = FIRST + decltype(i)::value;
      if constexpr (!EARLY && U + kAhead == F_K) v_here();
      fetch(std::integral_constant<int, U + kAhead>{});
      const T8 x = op[U % (kAhead + 1)];
      if constexpr (U < F_K) {
        constexpr int kb = U / KK, kk = U % KK;
        if constexpr (kk == KK - 2 && kb + 1 < NKB) begin(std::integral_constant<int, kb + 1>{});
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) n[qb][kb] = mma(x, qf[qb][kk], n[qb][kb]);
      } else {
        constexpr int f = (U - F_K) / MB, mb = (U - F_K) % MB;
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) o[qb][mb] = mma(x, __builtin_bit_cast(T8, p[qb][f]), o[qb][mb]);
      }
      if constexpr (NEXT) {
        static_for<3>([&](auto w) {   // the oldest first
          constexpr int W = 2 - decltype(w)::value, V = U - W * LAG;
          constexpr int P0 = V < 0 ? 0 : V < LAST ? V * PAIRS / LAST : PAIRS;
          constexpr int P1 = V < 0 ? 0 : V < LAST ? (V + 1) * PAIRS / LAST : PAIRS;
          // With LAG 0 the parts of one slot run in their own order.
          constexpr int R = LAG ? W : 2 - W;
          part(std::integral_constant<int, R>{}, std::integral_constant<int, P0>{}, std::integral_constant<int, P1>{});
        });
        // The next scores' maximum: evenly over the V slots but the first.
        if constexpr (U > F_K) {
          constexpr int E0 = (U - F_K - 1) * NKB * 16 / (F_V - 1), E1 = (U - F_K) * NKB * 16 / (F_V - 1);
#pragma unroll
          for (int qb = 0; qb < QB; ++qb) {
            if constexpr (E0 == 0) top[qb] = n[qb][0][0];
#pragma unroll
            for (int e = E0; e < E1; ++e) top[qb] = fmaxf(top[qb], n[qb][e / 16][e % 16]);
            pin(top[qb]);
          }
        }
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) {
          pin(sum[qb][0]);
          pin(sum[qb][1]);
        }
      }
      if constexpr (NEXT) beside(std::integral_constant<int, U>{});
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) l[qb] += sum[qb][0] + sum[qb][1];
  };

  // Tile j lies in buffers j % RB.
  //
  // Shared tiles: a barrier every SP steps (two where LDS has room, since a
  // barrier is a wait for the slowest of four waves); behind that of step j every
  // wave has left K tile j, V tile j - 1 and those before, and their buffers take
  // the next SP tiles.
  // Own tiles: a buffer is refilled as soon as its wave has read it, so that
  // three of the four are always on their way (the read of k and v is what such
  // a call spends its time on): K tile j + 3 between the products of step j, V
  // tile j + 2 after them. A tile past the last is asked for too, which writes
  // zeros and keeps the counts.
  uint64_t early[RB] = {};   // of the first tiles
  auto row_tile = [&](const int rt, const bool again, const bool another) {
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    m[qb] = -FLT_MAX;
    l[qb] = 0.f;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[qb][mb][e] = 0.f;
  }
  if (nt > 0) {
    Scores s0, s1;
    float top[QB];
    constexpr int SP = G::SP;
    int j = 0;
    uint64_t bits[SP + 1] = {};   // of tiles j + SP .. j + 2 SP; own tiles: bits[0] of j + 2
    auto none = [](auto...) {};
    // Scores of tile j + 1 into n beside the rest of tile j; u = j % RB.
    auto advance = [&](auto u, const Scores &s, Scores &n) {
      constexpr int B = decltype(u)::value;
      if constexpr (SHARED) {
        if constexpr (RESIDENT) {
          // All tiles came with the first row tile's.
          if (B == 0 && !again) arrived(std::integral_constant<int, 0>{});
          bits[SP == 1 ? 1 : B % SP] = B + 2 < RB ? early[B + 2] : 0;
        } else if constexpr (B % SP == 0) {
          arrived(std::integral_constant<int, 0>{});
          if (MASK && j == 0) bits[SP] = seen(2 * SP);
        }
        set_bias(B % 2, bits[SP == 1 ? 1 : B % SP]);   // of tile j + 2
        // The next SP tiles' bits: read before the step, voted on after it.
        constexpr bool VOTE = MASK && !RESIDENT && B % SP == SP - 1;
        uint8_t bytes[SP];
        if constexpr (VOTE) {
#pragma unroll
          for (int i = 0; i < SP; ++i) bytes[i] = mask_byte(j + SP + 2 + i);
        }
        step(u, std::integral_constant<int, 1>{}, s, n, top, none, [&](auto slot) {
          // In slots 1, 3, ...: V tiles j + SP .., K tiles j + SP + 1 .., the masks.
          constexpr int U = decltype(slot)::value, I = U / 2;
          if constexpr (!RESIDENT && B % SP == 0 && U % 2 == 1) {
            if constexpr (I < SP) {
              if (j > 0) issue_v(j + SP + I, (B + SP + I) % RB, bits[I]);
            } else if constexpr (I < 2 * SP) {
              constexpr int K = I - SP + 1;
              if (j > 0 || K == SP) issue_k(j + SP + K, (B + SP + K) % RB, bits[K]);
            }
            if constexpr (I == 2 * SP - 1) {
#pragma unroll
              for (int i = 1; i <= SP; ++i) issue_mask(j + 3 * SP + i);
            }
          }
        });
        if constexpr (VOTE) {
          bits[0] = bits[SP];
#pragma unroll
          for (int i = 0; i < SP; ++i) bits[1 + i] = vote(j + SP + 2 + i, bytes[i]);
        }
      } else {
        uint64_t next = 0;
        arrived(std::integral_constant<int, 3 * NI + MASK>{});
        step(u, std::integral_constant<int, 1>{}, s, n, top,
             [&] { arrived(std::integral_constant<int, 2 * NI + MASK>{}); },
             [&](auto slot) {
               if constexpr (decltype(slot)::value == F_K - 1) {   // the K tile's last use
                 next = seen(j + 3);
                 set_bias((B + 1) % 2, next);
                 issue_mask(j + 5);
                 issue_k(j + 3, (B + 3) % RB, next);
               }
             });
        issue_v(j + 2, B, bits[0]);
        bits[0] = next;
      }
      cut(n, j + 1, top);
      follow(top);
      ++j;
    };
    // The first tiles: every buffer is asked for at once, so that a short row of
    // keys costs one trip to memory.
    if (!again) {
    if constexpr (MASK) {
#pragma unroll
      for (int i = 0; i < (SHARED ? RB : 4); ++i) issue_mask(i);
      arrived(std::integral_constant<int, 0>{});
#pragma unroll
      for (int i = 0; i < RB; ++i) early[i] = seen(i);
      if constexpr (!SHARED) bits[0] = seen(2);
      else if constexpr (!RESIDENT) {
#pragma unroll
        for (int i = 0; i < SP; ++i) bits[i] = early[SP + i];
#pragma unroll
        for (int i = 0; i <= SP; ++i) issue_mask(RB + i);
      }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) issue_k(i, i, early[i]);
#pragma unroll
    for (int i = 0; i < (SHARED ? RB : 1); ++i) issue_v(i, i, early[i]);
    arrived(std::integral_constant<int, (RB - 1 + (SHARED ? RB : 1)) * NI>{});
    }
    take_q();
    if (another) load_q(rt + 1);
    set_bias(0, early[0]);
    set_bias(1, early[1]);
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
      const floatx16 init = start(0, kb);
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) s0[qb][kb] = init;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const T8 x = k_operand(0, kb * KK + kk);
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) s0[qb][kb] = mma(x, qf[qb][kk], s0[qb][kb]);
      }
    }
    if constexpr (!SHARED) {
      set_bias(0, bits[0]);
      issue_mask(4);
      issue_k(2, 0, bits[0]);
      issue_v(1, 1, early[1]);
    }
    maximum(s0, top);
    cut(s0, 0, top);
    follow(top);
    bool more = nt > 1;
    while (more) {
      static_for<RB>([&](auto u) {
        if (!more) return;
        if constexpr (decltype(u)::value % 2 == 0) advance(u, s0, s1);
        else advance(u, s1, s0);
        more = j + 1 < nt;
        if constexpr (decltype(u)::value % 2 == 0) {
          if (!more) {
#pragma unroll
            for (int qb = 0; qb < QB; ++qb)
#pragma unroll
              for (int kb = 0; kb < NKB; ++kb) s0[qb][kb] = s1[qb][kb];
          }
        }
      });
    }
    step(j % RB, std::integral_constant<int, 0>{}, s0, s1, top,
         [&] {
           if (!again) arrived(std::integral_constant<int, SHARED ? 0 : 2 * NI>{});
         },
         none);
    // The tiles past the last: LDS is used again below, and by the next workgroup.
    if constexpr (!SHARED) arrived(std::integral_constant<int, 0>{});
  }

  // No key was seen: nothing is added, whatever q holds. (An infinite q times the
  // zeros in place of a row that was not fetched is NaN, and its p with it.)
  if constexpr (MASK) {
    if (visible == 0) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) {
        m[qb] = -FLT_MAX;
        l[qb] = 0.f;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[qb][mb][e] = 0.f;
      }
    }
  }

  // ---- Results: lane = row n32, elements 32 mb + 8 a + 4 half + (0..3) of o.
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) l[qb] = sum_halves(l[qb]);
  if constexpr (SHARED) {
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      const int tr = wave * 32 * QB + qb * 32 + n32, r = rt * ROWS + tr;
      const float inv = l[qb] == 0.f ? 0.f : 1.f / l[qb];
      if (a.splits > 1) {
        const int64_t at = ((int64_t)g * a.row_tiles + rt) * ROWS + tr;
        if (r < a.rows) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int e = 32 * mb + 8 * u + 4 * half;
              if (e < a.d) {
                floatx4 f;
#pragma unroll
                for (int x = 0; x < 4; ++x) f[x] = o[qb][mb][4 * u + x] * inv;
                *reinterpret_cast<floatx4 *>(a.part + at * a.d + e) = f;
              }
            }
          if (half == 0) a.part_lse[at] = l[qb] == 0.f ? -INFINITY : m[qb] + __log2f(l[qb]);
        }
      } else {
        const int i = divide(r, a.by_group), h = hk * a.group + r - i * a.group;
        T *p = static_cast<T *>(a.out) + b * a.os[0] + i * a.os[1] + h * a.os[2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            // Halves of 8 elements lie in the two lane halves: swap, so that lane
            // half h has all of chunk u + h.
            unsigned w[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const F2 f = {o[qb][mb][4 * (u + x) + 2 * y] * inv, o[qb][mb][4 * (u + x) + 2 * y + 1] * inv};
                w[x][y] = __builtin_bit_cast(unsigned, __builtin_convertvector(f, T2));
              }
            const auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            const int e = 32 * mb + 8 * (u + half);
            if (r < a.rows && e < a.d) *reinterpret_cast<uintx4 *>(p + e) = uintx4{s0[0], s1[0], s0[1], s1[1]};
          }
        if (a.lse && r < a.rows && half == 0)
          a.lse[((int64_t)b * a.hq + h) * a.lq + i] =
              l[qb] == 0.f ? -INFINITY : (m[qb] + __log2f(l[qb])) * 0.69314718055994531f;
      }
    }
  } else {
    // Join the waves: out = sum_w 2^(M_w - M) O_w / sum_w 2^(M_w - M) l_w.
    float *jo = reinterpret_cast<float *>(lds), *jm = jo + NW * 32 * G::JOIN_PITCH, *jl = jm + NW * 32;
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        floatx4 f;
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = o[0][mb][4 * u + x];
        *reinterpret_cast<floatx4 *>(jo + (wave * 32 + n32) * G::JOIN_PITCH + 32 * mb + 8 * u + 4 * half) = f;
      }
    if (half == 0) {
      jm[wave * 32 + n32] = m[0];
      jl[wave * 32 + n32] = l[0];
    }
    __syncthreads();
    const int chunks = a.d / 8;
    for (int it = threadIdx.x; it < 32 * chunks; it += NW * 64) {
      const int tr = it / chunks, e = (it % chunks) * 8, r = rt * ROWS + tr;
      if (r >= a.rows) break;   // rows only grow with it
      float top = jm[tr], sum = 0.f, f[8] = {};
#pragma unroll
      for (int w = 1; w < NW; ++w) top = fmaxf(top, jm[w * 32 + tr]);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float x = __builtin_amdgcn_exp2f(jm[w * 32 + tr] - top);
        sum += x * jl[w * 32 + tr];
#pragma unroll
        for (int y = 0; y < 8; ++y) f[y] += x * jo[(w * 32 + tr) * G::JOIN_PITCH + e + y];
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);
#pragma unroll
      for (int y = 0; y < 8; ++y) f[y] *= inv;
      if (a.splits > 1) {
        const int64_t at = ((int64_t)g * a.row_tiles + rt) * ROWS + tr;
        floatx4 *p = reinterpret_cast<floatx4 *>(a.part + at * a.d + e);
        p[0] = floatx4{f[0], f[1], f[2], f[3]};
        p[1] = floatx4{f[4], f[5], f[6], f[7]};
        if (e == 0) a.part_lse[at] = lse2;
      } else {
        const int i = divide(r, a.by_group), h = hk * a.group + r - i * a.group;
        T8 w;
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y] = (T)f[y];
        *reinterpret_cast<T8 *>(static_cast<T *>(a.out) + b * a.os[0] + i * a.os[1] + h * a.os[2] + e) = w;
        if (a.lse && e == 0) a.lse[((int64_t)b * a.hq + h) * a.lq + i] = lse2 * 0.69314718055994531f;
      }
    }
  }
  };
  if constexpr (RESIDENT) {
    const int rt1 = min(rt0 + a.run, a.row_tiles);
    for (int rt = rt0; rt < rt1; ++rt) row_tile(rt, rt > rt0, rt + 1 < rt1);
  } else {
    row_tile(rt0, false, false);
  }
}

constexpr int kHeads[] = {32, 64, 96, 128, 160, 192, 256};   // padded head sizes

// Calls f(std::integral_constant<int, DP>) for the plan's padded head size.
template <typename F>
hipError_t for_head(int dp, F &&f) {
  switch (dp) {
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 96: return f(std::integral_constant<int, 96>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 160: return f(std::integral_constant<int, 160>{});
    case 192: return f(std::integral_constant<int, 192>{});
    default: return f(std::integral_constant<int, 256>{});
  }
}

constexpr int kResidentHead = 128;   // the largest padded head with a RESIDENT form
constexpr int few_waves(int dp) { return dp <= 128 ? 4 : 2; }

int64_t join_items(const AttentionPlan &p) { return (int64_t)p.d.n * p.d.hkv * p.rows * (p.d.d / 8); }

template <typename T>
hipError_t launch_t(const AttentionPlan &p, const Args &a, hipStream_t s) {
  const unsigned blocks = (unsigned)((int64_t)a.groups * a.runs);
  hipError_t e = for_head(p.dp, [&](auto dp) -> hipError_t {
    constexpr int DP = decltype(dp)::value;
    auto go = [&](auto waves, auto shared, auto resident) -> hipError_t {
      constexpr int NW = decltype(waves)::value;
      constexpr bool S = decltype(shared)::value, R = decltype(resident)::value;
      return a.mask ? launch_kernel(is_k11_attention<T, DP, 1, NW, S, R, true>, dim3(blocks), dim3(NW * 64), 0, s, a)
                    : launch_kernel(is_k11_attention<T, DP, 1, NW, S, R, false>, dim3(blocks), dim3(NW * 64), 0, s, a);
    };
    using four = std::integral_constant<int, 4>;
    if (p.tile_rows == 32) return go(std::integral_constant<int, few_waves(DP)>{}, std::false_type{}, std::false_type{});
    if constexpr (DP <= kResidentHead)
      if (p.run > 1) return go(four{}, std::true_type{}, std::true_type{});
    return go(four{}, std::true_type{}, std::false_type{});
  });
  if (e != hipSuccess || p.splits == 1) return e;
  JoinArgs j = {a.part, a.part_lse, a.out, a.lse, {a.os[0], a.os[1], a.os[2]}, a.lq, a.hq, a.hkv, a.d, a.group, a.rows,
                a.row_tiles, p.tile_rows, p.splits, join_group(p.splits), join_items(p)};
  return launch_join<T>(j, s);
}

}  // namespace

// How a call is cut, by an estimate of its time in microseconds fitted to runs of
// 1024 and 4096 keys with 9 entries x heads of 1021 to 4000 queries, heads of 32 to 256
// (within 15%), and the read of k and v where that takes longer:
//   shared tiles, 128 rows a workgroup, a step of 64 keys: 0.50 + dp / 350 alone
//     on its CU, 0.70 + dp / 140 for two (heads of 64: 0.68 and 1.1 measured; of
//     128: 0.86 and 1.5); heads over 128 leave LDS for one, 0.1 + dp / 140;
//   own tiles, 32 rows, a step of 32 keys a wave: 0.60 + dp / 500 (heads of 96:
//     0.75 measured) alone, half as much again for two (heads to 64);
//   start and end: 5 + dp / 32 (shared), 5 + dp / 64 (own);
//   joining splits: 1.5, and their 32-bit results written and read at 4 TB/s.
// E.g. 2042 rows x 9 heads of 96 over 1543 keys: shared, no splits, 27.4 us; three
// splits 33.2; own tiles 43.8. 800 rows: own tiles 16.9; shared in two 21.9.
struct Cut {
  bool few;
  int splits, split_keys;
  double us;
};

Cut estimate(const AttentionPlan &p, bool few, int64_t splits) {
  const cross_attention_desc &d = p.d;
  const int step = few ? 32 * few_waves(p.dp) : 64;
  const int64_t heads = (int64_t)d.n * d.hkv;
  if (p.rows <= 0 || heads <= 0) return {few, 1, step, 0.0};
  const int64_t units = heads * ((p.rows + (few ? 31 : 127)) / (few ? 32 : 128));
  const int tile = few ? 32 : 64;
  int64_t keys = ((d.lk + splits - 1) / splits + tile - 1) / tile * tile;
  if (keys < tile) keys = tile;
  Cut c = {few, (int)((d.lk + keys - 1) / keys), (int)keys, 0.0};
  if (c.splits < 1) c.splits = 1;
  const int64_t blocks = units * c.splits;
  const bool pairs = few ? p.dp <= 64 : p.dp <= 128;      // two workgroups on a CU
  const double one = few ? 0.6 + p.dp / 500.0 : pairs ? 0.5 + p.dp / 350.0 : 0.1 + p.dp / 140.0;
  const double two = few ? 1.5 * one : 0.7 + p.dp / 140.0;
  const int64_t round = pairs ? 512 : 256;
  const int64_t rest = blocks % round;
  const double per_step = (double)(blocks / round) * (pairs ? two : one) +
                          (rest == 0 ? 0.0 : rest > 256 ? two : one);
  const double read = (double)heads * d.lk * d.d * 4.0 / 5.0e6;   // of k and v at 5 TB/s
  const double walk = (double)((keys + step - 1) / step) * per_step;
  // The shorter of the two is not quite hidden by the longer.
  c.us = 5.0 + p.dp / (few ? 64.0 : 32.0) + (walk > read ? walk + read / 4 : read + walk / 4);
  if (c.splits > 1) c.us += 1.5 + 8.0 * (double)heads * p.rows * c.splits * d.d / 4.0e6;
  return c;
}

bool configure_attention(AttentionPlan &p) {
  const cross_attention_desc &d = p.d;
  p.group = d.hq / d.hkv;
  p.rows = d.lq * p.group;
  p.dp = kHeads[0];
  for (const int h : kHeads)
    if (p.dp < d.d) p.dp = h;
  Cut best = estimate(p, p.rows <= 32, 1);
  for (int kind = 0; kind < 2; ++kind)
    for (int64_t splits = 1; splits <= 128 && splits * 128 <= d.lk + 127; splits += splits < 16 ? 1 : splits / 8) {
      if (kind == 1 && p.rows <= 32) break;   // a shared tile would leave waves without rows
      if (splits > 1 && (double)(join_items(p) << join_group((int)splits)) + 255.0 > kMaxThreads) break;
      const Cut c = estimate(p, kind == 0, splits);
      if (c.us < best.us) best = c;
    }
  const bool few = best.few;
  p.tile_rows = few ? 32 : 128;
  p.row_tiles = (p.rows + p.tile_rows - 1) / p.tile_rows;
  p.block = few ? 64 * few_waves(p.dp) : 256;
  p.units = (int64_t)d.n * d.hkv * p.row_tiles;
  p.splits = best.splits;
  p.split_keys = best.split_keys;
  // Few keys and many row tiles: a workgroup keeps the keys for several, which
  // leaves one round of workgroups. (One tile each: the trip to memory, the
  // products and the stores of one row tile follow each other in every workgroup;
  // 8 x 4096 rows x 8 heads of 40 over 120 keys: 25.8 us against 18.4.)
  const int kept = p.dp <= 64 ? 4 : 2;   // tiles that fit the buffers
  p.run = 1;
  if (!few && p.splits == 1 && p.dp <= kResidentHead && d.lk <= kept * 64) {
    const int64_t run = p.units / 512;
    p.run = (int)(run < 1 ? 1 : run > p.row_tiles ? p.row_tiles : run);
  }
  p.name = few ? "is_k11_attention (own tiles)" : p.run > 1 ? "is_k11_attention (resident)" : "is_k11_attention";
  p.workgroups = (int64_t)d.n * d.hkv * ((p.row_tiles + p.run - 1) / p.run);
  (void)for_head(p.dp, [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    p.lds = few ? Geo<DP, few_waves(DP), false, false>::BYTES : Geo<DP, 4, true, false>::BYTES;
    return hipSuccess;
  });
  return (double)p.workgroups * p.splits * p.block <= kMaxThreads;
}

size_t attention_workspace(const AttentionPlan &p) {
  return p.splits == 1 ? 0 : (size_t)p.units * p.splits * p.tile_rows * (p.d.d + 1) * 4;
}

hipError_t launch_attention(const AttentionPlan &p, const void *q, const void *k, const void *v,
                            const uint8_t *mask, const int32_t *lengths, void *out, float *lse, void *ws,
                            hipStream_t s) {
  const cross_attention_desc &d = p.d;
  Args a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.mask = mask;
  a.lengths = lengths;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float *>(ws);
  a.part_lse = a.part ? a.part + (size_t)p.units * p.splits * p.tile_rows * d.d : nullptr;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = d.q_stride[i];
    a.ks[i] = d.k_stride[i];
    a.vs[i] = d.v_stride[i];
    a.os[i] = d.out_stride[i];
  }
  // One key has no next one: its stride may be anything, and the kernel forms the
  // span of a whole tile from it in 32 bits.
  if (d.lk <= 1) a.ks[1] = a.vs[1] = 0;
  a.mask_bs = d.mask_batch_stride;
  a.lq = d.lq;
  a.lk = d.lk;
  a.hq = d.hq;
  a.hkv = d.hkv;
  a.d = d.d;
  a.group = p.group;
  a.rows = p.rows;
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.split_keys = p.split_keys;
  a.groups = d.n * d.hkv * p.splits;
  a.run = p.run;
  a.runs = (p.row_tiles + p.run - 1) / p.run;
  a.by_group = divisor((unsigned)p.group);
  a.by_runs = divisor((unsigned)a.runs);
  a.by_splits = divisor((unsigned)p.splits);
  a.by_hkv = divisor((unsigned)d.hkv);
  a.flip = p.scale < 0.f ? 0x80008000u : 0u;
  a.c = score_factor(p.scale);
  return d.dtype == IS_F16 ? launch_t<_Float16>(p, a, s) : launch_t<__bf16>(p, a, s);
}

}  // namespace is
