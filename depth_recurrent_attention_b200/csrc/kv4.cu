// A 4-bit cache of attention keys and values: rows quantised as they are written, read back,
// and attended by one query token a sequence.
//
// A group is KV4_GROUP = 64 consecutive channels of one head of one token:
//   s = bf16((max - min) / 15), m = bf16(min), c = min(max(rint((x - m) / s), 0), 15), c = 0
//   where s = 0; the value held is s c + m.  A group with a NaN or a magnitude above 2^100
//   holds s = m = NaN and reads back as NaN (below, no sum of the attention overflows).
// 64 + 8 bits of pairs in 64 channels: 0.5625 bytes a value, 3.6 times fewer than bf16.
//
// Blocks of 64 tokens lie contiguously: K codes [ng][64][32 bytes], V codes, K pairs [ng][64]
// (bf16 s, bf16 m), V pairs, ng = d / 64: one bulk copy brings a block into shared memory, and
// a 32-byte code row of a plane is one sector.  Channel 2i of a plane's row is the low half of
// byte i.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/dreamer.h"
#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace dreamer {
namespace ops {
namespace {

constexpr int PLANE = KV4_BLOCK * 32;  // bytes of a code plane of a block
constexpr int PAIRS = KV4_BLOCK * 4;   // bytes of a pair plane of a block

// ---- rows in and out -------------------------------------------------------------------
// A CTA takes ROWS rows and eight (head, plane) pairs of the keys or of the values (blockIdx.z), a
// warp one of the eight: 8 lanes hold a group's 64 channels, so a warp step is four consecutive
// rows of one (head, plane), 128-byte reads, and 128 contiguous bytes of codes and 16 of pairs
// where the rows are neighbours in a block.  64 rows a CTA where that still fills the GPU (the search
// for the rows' places is paid once a CTA; 32 and 128 measured 2 and 9 % slower), else 16.
//
// The store is bound by instructions (about 180 a step of 4 rows x 64 channels), the load by memory:
// 19198 rows of 16 heads of 128, keys and values, bfloat16, take 63 us (157 MB read, 44 written) and 40
// (44 read, 157 written); codes from 64-bit quotients took 141.
constexpr int CU_SMEM = 1024;  // boundaries searched in shared memory up to this many sequences

struct RowArgs {
  uint8_t *data;
  int B, Hkv, ng, cap;
  int limit;      // positions that may be used
  const void *k, *v;
  long ldk, ldv;
  const int *cu, *start;
  int n_rows;
  int zero_rest;  // load: rows of no sequence become zeros
  int *err;
};

// Place in the cache of the CTA's rows: byte offset of a row's codes in head 0's plane 0, and of its
// pair from there on.  Row r belongs to the sequence b with cu[b] <= r < cu[b + 1]; an offset below 0: the
// row is in no sequence, or its position is outside 0 .. limit - 1 (reported).
struct Place {
  long codes;
  int pair;
};
template <int ROWS>
__device__ __forceinline__ void find_slots(const RowArgs &a, int row0, int *scu, Place *place) {
  const int tid = threadIdx.x;
  const int *cu = a.cu;
  if (a.cu && a.B <= CU_SMEM) {
    for (int i = tid; i <= a.B; i += blockDim.x) scu[i] = a.cu[i];
    cu = scu;
  }
  __syncthreads();
  if (tid < ROWS) {
    const int r = row0 + tid;
    int p = -1, b = -1;
    long off = 0;
    if (r < a.n_rows) {
      if (!a.cu) {
        b = r;
      } else {
        int lo = 0, hi = a.B;  // first b whose end cu[b + 1] lies past r
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (cu[mid + 1] > r) hi = mid;
          else lo = mid + 1;
        }
        if (lo < a.B && cu[lo] <= r) {
          b = lo;
          off = (long)r - cu[lo];
        }
      }
      if (b >= 0) {
        const long q = a.start[b] + off;
        if (q >= 0 && q < a.limit) p = (int)q;
        else raise_dev_error(a.err, DEV_BAD_INDEX);
      }
    }
    const int t = p % KV4_BLOCK;
    place[tid].codes = p < 0 ? -1 : ((long)b * a.Hkv * (a.cap / KV4_BLOCK) + p / KV4_BLOCK) * (a.ng * 2 * (PLANE + PAIRS)) + t * 32;
    place[tid].pair = 2 * a.ng * PLANE - t * (32 - 4);
  }
  __syncthreads();
}

// Eight consecutive values as they were read
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float *p) { load8(p, v); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = 0.f;
  }
  // the largest value and the largest negated value of the group's 8 lanes; NaN where one is
  __device__ __forceinline__ void range(float &mx, float &neg) const {
    mx = v[0];
    neg = -v[0];
#pragma unroll
    for (int e = 1; e < 8; e++) {
      mx = max_nan(mx, v[e]);
      neg = max_nan(neg, -v[e]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      neg = max_nan(neg, __shfl_xor_sync(0xffffffffu, neg, o));
    }
  }
  static __device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ float value(int e) const { return v[e]; }
  __device__ __forceinline__ float minus(int e, float m) const { return v[e] - m; }
};
template <> struct Raw8<bf16> {
  uint32_t u[4];
  __device__ __forceinline__ void load(const bf16 *p) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    u[0] = w.x; u[1] = w.y; u[2] = w.z; u[3] = w.w;
  }
  __device__ __forceinline__ void zero() { u[0] = u[1] = u[2] = u[3] = 0; }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ void range(float &mx, float &neg) const {
    const uint32_t hi = max2(max2(u[0], u[1]), max2(u[2], u[3]));
    const uint32_t lo = min2(min2(u[0], u[1]), min2(u[2], u[3])) ^ 0x80008000u;
    // (max, max of the negated) in the two halves of a word
    uint32_t r = max2(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) r = max2(r, __shfl_xor_sync(0xffffffffu, r, o));
    mx = __uint_as_float(r << 16);
    neg = __uint_as_float(r & 0xffff0000u);
  }
  __device__ __forceinline__ float value(int e) const {
    return __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
  }
  // x - m rounded once, the bf16 half taken as it is
  __device__ __forceinline__ float minus(int e, float m) const {
    float d;
    if (e & 1)
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tfma.rn.f32.bf16 %0, h, %2, %3;\n\t}"
          : "=f"(d) : "r"(u[e >> 1]), "h"((unsigned short)0x3F80), "f"(-m));
    else
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tfma.rn.f32.bf16 %0, l, %2, %3;\n\t}"
          : "=f"(d) : "r"(u[e >> 1]), "h"((unsigned short)0x3F80), "f"(-m));
    return d;
  }
};

// c = min(max(rint((x - m) / s), 0), 15) of the exact quotient, the form in 64 bits
__device__ __noinline__ float code_exact(float x, float m, float s) {
  const double q = rint(((double)x - (double)m) / (double)s);
  return (float)fmin(fmax(q, 0.0), 15.0);
}
// (max - min) / 15 in 64 bits
__device__ __noinline__ float step_exact(float mx, float mn) { return (float)(((double)mx - (double)mn) / 15.0); }

// Eight codes of a lane's values, four bits each.  The quotient in 32 bits is off by less than 2^-18,
// so it rounds as the exact one does unless that lies within 2^-16 of a half, which the remainder
// d - c s (exact: at most 24 bits) shows.  There the remainder decides where d = x - m is
// exact, as it nearly always is for bfloat16 (a tie goes to the even code), else the form in 64 bits.
// bfloat16: m is the minimum itself and s within 2^-8 of a 15th, so quotients lie in 0 .. 15.06.
template <typename T>
__device__ __forceinline__ uint32_t codes8(const Raw8<T> &x, float m, float s) {
  constexpr bool CLAMP = sizeof(T) == 4;
  float inv;  // within 2^-23
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float near = s * (0.5f - 0x1p-16f);
  const uint64_t inv2 = f2_pack(inv, inv), s2 = f2_pack(s, s), magic2 = f2_pack(12582912.f, 12582912.f);
  const uint64_t minus1 = f2_pack(-1.f, -1.f);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint64_t d2 = f2_pack(x.minus(e, m), x.minus(e + 1, m));
    uint64_t n2;  // 1.5 * 2^23 + the rounded quotients, half to even
    bool in[2] = {true, true};
    if (CLAMP) {
      float2 y = f2_unpack(d2);
      y.x = fminf(fmaxf(y.x * inv, 0.f), 15.f);
      y.y = fminf(fmaxf(y.y * inv, 0.f), 15.f);
      in[0] = y.x > 0.f && y.x < 15.f;
      in[1] = y.y > 0.f && y.y < 15.f;
      n2 = f2_add(f2_pack(y.x, y.y), magic2);
    } else {
      n2 = f2_fma(d2, inv2, magic2);
    }
    const float2 t2 = f2_unpack(f2_fma(f2_fma(n2, minus1, magic2), s2, d2)), nn = f2_unpack(n2), dd = f2_unpack(d2);
    float n[2] = {nn.x, nn.y};
    const float t[2] = {t2.x, t2.y}, d[2] = {dd.x, dd.y};
#pragma unroll
    for (int k = 0; k < 2; k++) {
      if (fabsf(t[k]) >= near && in[k]) {
        const float v = x.value(e + k), h = 0.5f * s;
        if (d[k] + m == v && v - d[k] == m) {
          const bool odd = __float_as_uint(n[k]) & 1u;
          if (t[k] > h || (t[k] == h && odd)) n[k] += 1.f;
          else if (t[k] < -h || (t[k] == -h && odd)) n[k] -= 1.f;
        } else {
          n[k] = code_exact(v, m, s) + 12582912.f;
        }
      }
      w += __float_as_uint(n[k]) << (4 * (e + k));
    }
  }
  // the sum of 0x4B400000 << 4 e
  constexpr uint32_t base = 0x4B400000u + 0xB4000000u + 0x40000000u;
  return w - base;
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 5 : 4) kv4_store_kernel(RowArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int scu[CU_SMEM + 1];
  __shared__ Place place[ROWS];
  const int row0 = blockIdx.x * ROWS;
  find_slots<ROWS>(a, row0, scu, place);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hp = blockIdx.y * 8 + warp;  // head * ng + plane
  if (hp >= a.Hkv * a.ng) return;
  const int head = hp / a.ng, plane = hp % a.ng;
  const int side = blockIdx.z;
  const int sub = lane >> 3;
  const long ld = side ? a.ldv : a.ldk;
  const T *src = reinterpret_cast<const T *>(side ? a.v : a.k) + (long)hp * KV4_GROUP + (lane & 7) * 8 +
                 (long)(row0 + sub) * ld;
  const int block_bytes = a.ng * 2 * (PLANE + PAIRS);
  uint8_t *dst = a.data + (long)head * (a.cap / KV4_BLOCK) * block_bytes + (side * a.ng + plane) * PLANE + (lane & 7) * 4;
  const int pair_at = (side * a.ng + plane) * (PAIRS - PLANE);
  Raw8<T> next;
  next.zero();
  if (place[sub].codes >= 0) next.load(src);
#pragma unroll 1
  for (int r = 0; r < ROWS; r += 4) {
    const Raw8<T> x = next;
    const Place pl = place[r + sub];
    src += 4 * ld;
    if (r + 4 < ROWS && place[r + 4 + sub].codes >= 0) next.load(src);  // the next rows', in flight meanwhile
    float mx, neg;
    x.range(mx, neg);
    // s = bf16((max - min) / 15): in 32 bits off by 2 steps at most, so a rounding within 4 of a tie is
    // taken in 64
    float sf = (mx + neg) * (1.0f / 15.0f);
    if ((((__float_as_uint(sf) + 4u) & 0xffffu) - 0x8000u) <= 8u || sf < 0x1p-100f) sf = step_exact(mx, -neg);
    uint32_t pr = bf2_pack_rn(sf, -neg);
    // NaN, infinite, out of range
    if (!(fmaxf(mx, neg) <= 0x1p100f) || !(mx + neg >= 0.f)) pr = 0x7fff7fffu;
    const float s = __uint_as_float(pr << 16), m = __uint_as_float(pr & 0xffff0000u);
    uint32_t w = 0;
    if (s >= 0x1p-100f) {
      w = codes8<T>(x, m, s);
    } else if (s > 0.f) {
#pragma unroll
      for (int e = 0; e < 8; e++) w |= (uint32_t)code_exact(x.value(e), m, s) << (4 * e);
    }
    if (pl.codes >= 0) {
      uint8_t *q = dst + pl.codes;
      *reinterpret_cast<uint32_t *>(q) = w;
      if ((lane & 7) == 0) *reinterpret_cast<uint32_t *>(q + pair_at + pl.pair) = pr;
    }
  }
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(256) kv4_load_kernel(RowArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int scu[CU_SMEM + 1];
  __shared__ Place place[ROWS];
  const int row0 = blockIdx.x * ROWS;
  find_slots<ROWS>(a, row0, scu, place);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hp = blockIdx.y * 8 + warp;
  if (hp >= a.Hkv * a.ng) return;
  const int head = hp / a.ng, plane = hp % a.ng;
  const int side = blockIdx.z;
  T *dst = reinterpret_cast<T *>(const_cast<void *>(side ? a.v : a.k)) + (long)hp * KV4_GROUP + (lane & 7) * 8;
  const long ld = side ? a.ldv : a.ldk;
  const int sub = lane >> 3;
  const int block_bytes = a.ng * 2 * (PLANE + PAIRS), sp = side * a.ng + plane;
  const uint8_t *from = a.data + (long)head * (a.cap / KV4_BLOCK) * block_bytes + sp * PLANE;
#pragma unroll 1
  for (int r0 = 0; r0 < ROWS; r0 += 16) {
    uint32_t w[4], pr[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const Place pl = place[r0 + i * 4 + sub];
      in[i] = pl.codes >= 0;
      w[i] = pr[i] = 0;
      if (!in[i]) continue;
      const uint8_t *q = from + pl.codes;
      w[i] = *reinterpret_cast<const uint32_t *>(q + (lane & 7) * 4);
      pr[i] = *reinterpret_cast<const uint32_t *>(q + pl.pair + sp * (PAIRS - PLANE));
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int r = row0 + r0 + i * 4 + sub;
      if (!in[i] && !(a.zero_rest && r < a.n_rows)) continue;
      const float s = __uint_as_float(pr[i] << 16), m = __uint_as_float(pr[i] & 0xffff0000u);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; e++) x[e] = fmaf(s, (float)((w[i] >> (4 * e)) & 15u), m);
      store8(dst + (long)r * ld, x);
    }
  }
}

// ---- attention of one query token a sequence over the cache ------------------------------
// A warp takes whole 64-token blocks, brought in by bulk copies into a ring of its own (4608 bytes at
// head dim 64, two or three in flight a warp), and
// multiplies on warp-level matrix instructions with the codes as the A operand:
//   scores   A = 16 keys x channels of K codes, B = channels x 8 columns of q
//   output   A = 16 channels x 16 keys of V codes, B = keys x 8 columns of weights
// What bounds it is turning nibbles into operands (the integer pipe), so
//   - bfloat16 runs on 8-bit integer products (m16n8k32): one mask makes four codes a word (the high
//     halves of bytes enter as 16 c).
//     q enters as a 16-bit fixed-point number of its plane's largest |q|, in two signed bytes (three where
//     two would move a score by more than 2^-10: a channel far above the others, large queries), a weight
//     p s as one of its column's largest in the block, in two unsigned bytes; the integer sums are
//     exact.  The steps are 2^-15 and 2^-16 of the largest (half a step of bf16 is 2^-8 of the value
//     itself, so q keeps its bf16 precision down to 1/128 of its plane's largest);
//   - float32 takes a code as the bf16 number c - 8, exact ((0x4300 | c) is 128 + c), and its operands
//     in three bf16 terms.
// With value = s c + m a score is s (q . c) + m sum(q), and the offsets enter the output as one sum of
// p m a plane.
// A column is (16-key tile of a supertile, query head): GP = 2, 4 or 8 columns hold the query heads
// that share a key head, and 8 / GP key tiles share one accumulator, each with q in its own columns
// and zeros elsewhere.  So one exponential a (key, query head) is computed also where a key head has
// one query head (GP = 2: one idle column of two).  Every column keeps its own running maximum and
// sum; they join at the end of a (sequence, key head): lanes, then warps.
//
// The rows r of a 16-key tile are the keys perm_row(r): with it a warp's 8-byte reads of K rows and
// 4-byte reads of V rows meet every bank once.
//
// Measured: the decode workload's depth (64 sequences of 4096 tokens, 16 heads of 64, 302 MB) 53 us replayed
// from a graph (5.7 TB/s), 60 a call among others (5.0), with the cluster form at one CTA an item; products
// on bf16 numbers instead of bytes took 82.  float32 (three terms): 122.
struct AttnArgs {
  const uint8_t *data;
  int B, Hkv, cap, Hq, G, qchunks;
  int limit;     // keys that a sequence may have
  const void *q;
  long ldq;
  void *out;
  long ldo;
  const int *lens;
  int len_add;
  float scale_log2;
  int *err;
  float *part;   // split form: [slot][GP][D + 4] partial outputs, maximum, sum
  int n_warps;   // split form: warps of the grid
#ifdef DREAMER_TEST_HOOKS
  Withhold withhold;
#endif
};

__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// unsigned bytes times signed (SB) or unsigned bytes, 32-bit integer sums: d = c + a b
template <bool SB>
__device__ __forceinline__ void mma16832(int *d, const uint32_t *a, uint32_t b0, uint32_t b1, const int *c) {
  if constexpr (SB)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
}
// transpose of an 8 x 8 matrix of 16-bit values held as mma fragments
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// nibbles j and j + 4 of w as the bf16 pair (c - 8, c' - 8)
template <int J> __device__ __forceinline__ uint32_t codes2(uint32_t w) {
  const uint32_t b = ((w >> (4 * J)) & 0x000f000fu) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(b), "r"(0x43084308u));
  return r;
}
__device__ __forceinline__ int perm_row(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 2) : g >> 1; }
__device__ __forceinline__ float2 pair_at(const uint8_t *p) {
  const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// An integer sum below 2^22 in magnitude, started at MAGIC, read as a float is 1.5 * 2^23 + sum.
constexpr int MAGIC = 0x4B400000;
constexpr float MAGIC_F = 12582912.f;

// The attention of one warp over blocks of one (sequence, key head) for up to GP query heads.
template <typename T, int NG, int GP>
struct WarpAttn {
  static constexpr bool INT = sizeof(T) == 2;       // products on bytes (else in three bf16 terms)
  static constexpr int D = NG * 64;
  static constexpr int NTI = 8 / GP;                // key tiles that share an accumulator
  static constexpr int NSUP = 4 / NTI;              // accumulators of a block
  static constexpr int QR = INT ? 8 : 24;           // registers of q a plane
  static constexpr int BLK = NG * 2 * (PLANE + PAIRS);  // bytes of a block

  uint32_t qf[NG][QR];
  float qs[NG][2];     // sum(q) of this lane's columns 2t, 2t + 1, times scale_log2
  float qi[NG][2];     // INT: the columns' fixed-point step, times scale_log2
  float o[NG][4][4];   // [plane][channel tile][c]: c >> 1 channel, c & 1 column 2t or 2t + 1
  float ofs[NG][2];    // sum of p m (of p (m + 8 s) where codes enter as c - 8)
  float m2[2], l2[2];
  uint32_t sel[NTI];   // 1 for the tile of column g, else 0
  // INT: are two bytes of q enough?  A rounded q is off by 0.29 steps, a code is
  // 8.7 (root mean squares), so a score of 64 channels is off by 20 s qi in log2; past 2^-10 (a weight off by
  // 6.8e-4; a bf16 output is by 1.7e-3 alone) the queries get a third byte.  64 sequences of 4096, 16 heads of
  // 64: 55 us with two bytes, 75 with three in every block (16 times larger queries).
  float q_max;         // largest |qi| of this lane's columns
  const T *qp;         // this lane's channels of column g's query head
  bool live;           // a column with a query head (else zeros)

  __device__ __forceinline__ void q_values(int p, float *v) const {
    load8(qp + p * 64, v);
    load8(qp + p * 64 + 8, v + 8);
#pragma unroll
    for (int e = 0; e < 16; e++)
      if (!live) v[e] = 0.f;
  }
  // What 127 * 256 steps of a query's plane are: its largest |q|, or 2^-110 (the step stays a normal number).
  // A q that is not finite leaves sum(q) so, and its scores with it.
  __device__ __forceinline__ float q_top(const float *v, bool &ok) const {
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e++) amax = fmaxf(amax, fabsf(v[e]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    ok = amax <= 0x1.fffffep127f;
    return ok ? fmaxf(amax, 0x1p-110f) : 1.f;
  }

  // q as B fragments: column g is query head g % GP; a lane holds channels 16 t .. 16 t + 15 of a plane
  __device__ __forceinline__ void start(const T *q, int nq, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int qh = g % GP;
#pragma unroll
    for (int ti = 0; ti < NTI; ti++) sel[ti] = g / GP == ti ? 1u : 0u;
    live = qh < nq;
    qp = q + (long)(live ? qh : 0) * D + 16 * t;
#pragma unroll
    for (int p = 0; p < NG; p++) {
      float v[16];
      q_values(p, v);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; e++) sum += v[e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int c0 = ((2 * t) % GP) * 4, c1 = ((2 * t + 1) % GP) * 4;
      qs[p][0] = __shfl_sync(0xffffffffu, sum, c0) * scale_log2;
      qs[p][1] = __shfl_sync(0xffffffffu, sum, c1) * scale_log2;
      if constexpr (INT) {
        bool ok;
        const float top = q_top(v, ok), step = top / 32512.f, inv = 32512.f / top;
        qi[p][0] = __shfl_sync(0xffffffffu, step, c0) * scale_log2;
        qi[p][1] = __shfl_sync(0xffffffffu, step, c1) * scale_log2;
        q_max = max3f(p == 0 ? 0.f : q_max, fabsf(qi[p][0]), fabsf(qi[p][1]));
#pragma unroll
        for (int w = 0; w < 4; w++) {  // even channels of the low 8, odd ones, then of the high 8
          uint32_t hi = 0, lo = 0;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int x = ok ? __float_as_int(fmaf(v[(w >> 1) * 8 + 2 * e + (w & 1)], inv, MAGIC_F)) - MAGIC : 0;
            const int h = (x + 128) >> 8;
            hi |= (uint32_t)(h & 255) << (8 * e);
            lo |= (uint32_t)((x - h * 256) & 255) << (8 * e);
          }
          qf[p][2 * w] = hi;
          qf[p][2 * w + 1] = lo;
        }
      } else {
        qi[p][0] = qi[p][1] = scale_log2;
#pragma unroll
        for (int w = 0; w < 2; w++)
#pragma unroll
          for (int j = 0; j < 4; j++) {  // the order of codes2<j> of word w: elements j and j + 4
            float lo = v[8 * w + j], hi = v[8 * w + j + 4];
#pragma unroll
            for (int k = 0; k < 3; k++) {
              const uint32_t pk = bf2_pack_rn(lo, hi);
              qf[p][(4 * w + j) * 3 + k] = pk;
              lo -= __uint_as_float(pk << 16);
              hi -= __uint_as_float(pk & 0xffff0000u);
            }
          }
      }
    }
#pragma unroll
    for (int c = 0; c < 2; c++) {
      m2[c] = -INFINITY;
      l2[c] = 0.f;
    }
#pragma unroll
    for (int p = 0; p < NG; p++) {
      ofs[p][0] = ofs[p][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < 4; mt++)
#pragma unroll
        for (int c = 0; c < 4; c++) o[p][mt][c] = 0.f;
    }
  }

  // an operand register in its own columns' tile, zero in the others: a product, which the busy integer
  // pipe does not see
  __device__ __forceinline__ uint32_t in_tile(uint32_t v, int ti) const {
    if constexpr (GP == 8) return v;
    uint32_t r;
    asm("mul.lo.u32 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(sel[ti]));
    return r;
  }

  // q . c (integer form: c; float form: c - 8) of supertile sp in plane p for this lane's two keys and
  // columns, to be scaled by qi and s
  __device__ __forceinline__ void products(const uint8_t *blk, int sp, int p, float *f) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t *kr = blk + p * PLANE + (sp * NTI * 16 + perm_row(g)) * 32 + 8 * t;
    if constexpr (INT) {
      // even channels (c) and odd ones (16 c: the high half of a byte as it lies) in sums of their own
      const int start[4] = {MAGIC, MAGIC, MAGIC, MAGIC};
      int he[4], le[4], ho[4], lo[4];
#pragma unroll
      for (int ti = 0; ti < NTI; ti++) {
        const uint2 w0 = *reinterpret_cast<const uint2 *>(kr + ti * 16 * 32);
        const uint2 w1 = *reinterpret_cast<const uint2 *>(kr + ti * 16 * 32 + 8 * 32);
        const uint32_t ev[4] = {w0.x & 0x0f0f0f0fu, w1.x & 0x0f0f0f0fu, w0.y & 0x0f0f0f0fu, w1.y & 0x0f0f0f0fu};
        const uint32_t od[4] = {w0.x & 0xf0f0f0f0u, w1.x & 0xf0f0f0f0u, w0.y & 0xf0f0f0f0u, w1.y & 0xf0f0f0f0u};
        mma16832<true>(he, ev, in_tile(qf[p][0], ti), in_tile(qf[p][4], ti), ti == 0 ? start : he);
        mma16832<true>(le, ev, in_tile(qf[p][1], ti), in_tile(qf[p][5], ti), ti == 0 ? start : le);
        mma16832<true>(ho, od, in_tile(qf[p][2], ti), in_tile(qf[p][6], ti), ti == 0 ? start : ho);
        mma16832<true>(lo, od, in_tile(qf[p][3], ti), in_tile(qf[p][7], ti), ti == 0 ? start : lo);
      }
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const float h = fmaf(0.0625f, __int_as_float(ho[c]) - MAGIC_F, __int_as_float(he[c]) - MAGIC_F);
        const float l = fmaf(0.0625f, __int_as_float(lo[c]) - MAGIC_F, __int_as_float(le[c]) - MAGIC_F);
        f[c] = fmaf(256.f, h, l);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; c++) f[c] = 0.f;
#pragma unroll
      for (int ti = 0; ti < NTI; ti++) {
        const uint2 w0 = *reinterpret_cast<const uint2 *>(kr + ti * 16 * 32);
        const uint2 w1 = *reinterpret_cast<const uint2 *>(kr + ti * 16 * 32 + 8 * 32);
        const bool on = GP == 8 || g / GP == ti;
        const uint32_t ww0[2] = {w0.x, w0.y}, ww1[2] = {w1.x, w1.y};
#pragma unroll
        for (int w = 0; w < 2; w++) {
          const uint32_t f0[4] = {codes2<0>(ww0[w]), codes2<0>(ww1[w]), codes2<1>(ww0[w]), codes2<1>(ww1[w])};
          const uint32_t f1[4] = {codes2<2>(ww0[w]), codes2<2>(ww1[w]), codes2<3>(ww0[w]), codes2<3>(ww1[w])};
#pragma unroll
          for (int k = 2; k >= 0; k--) {
            mma16816(f, f0, on ? qf[p][12 * w + k] : 0u, on ? qf[p][12 * w + 3 + k] : 0u);
            mma16816(f, f1, on ? qf[p][12 * w + 6 + k] : 0u, on ? qf[p][12 * w + 9 + k] : 0u);
          }
        }
      }
    }
  }

  // What rounding q to 16 bits left out of a block's scores: a third byte of every query
  __device__ __forceinline__ void scores_rest(const uint8_t *blk, int my_key, float (*x)[4]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 1
    for (int p = 0; p < NG; p++) {
      float v[16];
      q_values(p, v);
      bool ok;
      const float inv = 32512.f / q_top(v, ok);
      uint32_t b[4];
#pragma unroll
      for (int w = 0; w < 4; w++) {  // in the order of start(), in steps of 1/254 of its own: half of one is 127
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float u = v[(w >> 1) * 8 + 2 * e + (w & 1)], n = fmaf(u, inv, MAGIC_F) - MAGIC_F;
          r[e] = __float_as_uint(fmaf(fmaf(u, inv, -n), 254.f, MAGIC_F));
        }
        b[w] = ok ? __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410) : 0u;
      }
      const float i0 = (p == 0 ? qi[0][0] : qi[NG - 1][0]) * (1.f / 254.f);
      const float i1 = (p == 0 ? qi[0][1] : qi[NG - 1][1]) * (1.f / 254.f);
#pragma unroll
      for (int sp = 0; sp < NSUP; sp++) {
        const uint8_t *kr = blk + p * PLANE + (sp * NTI * 16 + perm_row(g)) * 32 + 8 * t;
        const int start[4] = {MAGIC, MAGIC, MAGIC, MAGIC};
        int he[4], ho[4];
#pragma unroll
        for (int ti = 0; ti < NTI; ti++) {
          const uint2 w0 = *reinterpret_cast<const uint2 *>(kr + ti * 16 * 32);
          const uint2 w1 = *reinterpret_cast<const uint2 *>(kr + ti * 16 * 32 + 8 * 32);
          const uint32_t ev[4] = {w0.x & 0x0f0f0f0fu, w1.x & 0x0f0f0f0fu, w0.y & 0x0f0f0f0fu, w1.y & 0x0f0f0f0fu};
          const uint32_t od[4] = {w0.x & 0xf0f0f0f0u, w1.x & 0xf0f0f0f0u, w0.y & 0xf0f0f0f0u, w1.y & 0xf0f0f0f0u};
          mma16832<true>(he, ev, in_tile(b[0], ti), in_tile(b[2], ti), ti == 0 ? start : he);
          mma16832<true>(ho, od, in_tile(b[1], ti), in_tile(b[3], ti), ti == 0 ? start : ho);
        }
        const uint8_t *kp = blk + 2 * NG * PLANE + p * PAIRS + (sp * NTI * 16 + my_key) * 4;
        const float s0 = pair_at(kp).x, s1 = pair_at(kp + 8 * 4).x;
        const float y[4] = {s0 * i0, s0 * i1, s1 * i0, s1 * i1};
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const float f = fmaf(0.0625f, __int_as_float(ho[c]) - MAGIC_F, __int_as_float(he[c]) - MAGIC_F);
          x[sp][c] = fmaf(y[c], f, x[sp][c]);
        }
      }
    }
  }

  // One block in shared memory: keys key0 .. key0 + 63, of which those below nkeys exist
  __device__ __forceinline__ void block(uint8_t *blk, int key0, int nkeys) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int my_key = ((2 * t) / GP) * 16 + perm_row(g);  // in a supertile: this lane's keys my_key (+ 8)
    const bool tail = key0 + KV4_BLOCK > nkeys;
    if (tail) {  // what lies behind the last key may be anything: its keys and values count as zero
      for (int k = lane; k < KV4_BLOCK; k += 32)
        if (key0 + k >= nkeys)
#pragma unroll
          for (int p = 0; p < 2 * NG; p++) *reinterpret_cast<uint32_t *>(blk + 2 * NG * PLANE + p * PAIRS + k * 4) = 0;
      tc::fence_proxy_async();  // the next copy into this stage comes after these writes
      __syncwarp();
    }
    float x[NSUP][4], smax = 0.f;
#pragma unroll
    for (int sp = 0; sp < NSUP; sp++) {
#pragma unroll
      for (int p = 0; p < NG; p++) {
        float f[4];
        products(blk, sp, p, f);
        const uint8_t *kp = blk + 2 * NG * PLANE + p * PAIRS + (sp * NTI * 16 + my_key) * 4;
        const float2 s0 = pair_at(kp), s1 = pair_at(kp + 8 * 4);
        if constexpr (INT) smax = max3f(smax, s0.x, s1.x);
        const float z0 = INT ? s0.y : fmaf(8.f, s0.x, s0.y), z1 = INT ? s1.y : fmaf(8.f, s1.x, s1.y);
        const float y0 = fmaf(s0.x * qi[p][0], f[0], z0 * qs[p][0]), y1 = fmaf(s0.x * qi[p][1], f[1], z0 * qs[p][1]);
        const float y2 = fmaf(s1.x * qi[p][0], f[2], z1 * qs[p][0]), y3 = fmaf(s1.x * qi[p][1], f[3], z1 * qs[p][1]);
        x[sp][0] = p == 0 ? y0 : x[sp][0] + y0;
        x[sp][1] = p == 0 ? y1 : x[sp][1] + y1;
        x[sp][2] = p == 0 ? y2 : x[sp][2] + y2;
        x[sp][3] = p == 0 ? y3 : x[sp][3] + y3;
      }
    }
    if constexpr (INT)
      if (__any_sync(0xffffffffu, smax * q_max > 0x1p-10f / 20.f)) scores_rest(blk, my_key, x);
    if (tail) {
#pragma unroll
      for (int sp = 0; sp < NSUP; sp++) {
        const int key = key0 + sp * NTI * 16 + my_key;
        if (key >= nkeys) x[sp][0] = x[sp][1] = -INFINITY;
        if (key + 8 >= nkeys) x[sp][2] = x[sp][3] = -INFINITY;
      }
    }
    // running maximum of the two columns, moved only when some score passes it by more than 2^8
    float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
    for (int sp = 1; sp < NSUP; sp++) {
      mx0 = max3f(mx0, x[sp][0], x[sp][2]);
      mx1 = max3f(mx1, x[sp][1], x[sp][3]);
    }
    if (__any_sync(0xffffffffu, mx0 > m2[0] + 8.f || mx1 > m2[1] + 8.f)) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, k));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, k));
      }
      const float n0 = fmaxf(m2[0], mx0), n1 = fmaxf(m2[1], mx1);
      const float a0 = m2[0] == -INFINITY ? 0.f : tc::ex2(m2[0] - n0);
      const float a1 = m2[1] == -INFINITY ? 0.f : tc::ex2(m2[1] - n1);
      m2[0] = n0;
      m2[1] = n1;
      l2[0] *= a0;
      l2[1] *= a1;
#pragma unroll
      for (int p = 0; p < NG; p++) {
        ofs[p][0] *= a0;
        ofs[p][1] *= a1;
#pragma unroll
        for (int mt = 0; mt < 4; mt++) {
          o[p][mt][0] *= a0;
          o[p][mt][1] *= a1;
          o[p][mt][2] *= a0;
          o[p][mt][3] *= a1;
        }
      }
    }
    {
      const float r0 = m2[0] == -INFINITY ? 0.f : m2[0], r1 = m2[1] == -INFINITY ? 0.f : m2[1];
#pragma unroll
      for (int sp = 0; sp < NSUP; sp++) {
        x[sp][0] = tc::ex2(x[sp][0] - r0);
        x[sp][1] = tc::ex2(x[sp][1] - r1);
        x[sp][2] = tc::ex2(x[sp][2] - r0);
        x[sp][3] = tc::ex2(x[sp][3] - r1);
        l2[0] += x[sp][0] + x[sp][2];
        l2[1] += x[sp][1] + x[sp][3];
      }
    }
#pragma unroll
    for (int p = 0; p < NG; p++) {
      if constexpr (INT) out_int(blk, p, my_key, x);
      else out_float(blk, p, my_key, x);
    }
  }

  // the four words (8 channels 8g .. 8g + 7 each) of a V tile's keys perm(2t), perm(2t + 1), (+ 8)
  __device__ __forceinline__ void v_words(const uint8_t *blk, int p, int tile, uint32_t *v) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t *vr = blk + (NG + p) * PLANE + tile * 16 * 32 + 4 * g;
    v[0] = *reinterpret_cast<const uint32_t *>(vr + perm_row(2 * t) * 32);
    v[1] = *reinterpret_cast<const uint32_t *>(vr + perm_row(2 * t + 1) * 32);
    v[2] = *reinterpret_cast<const uint32_t *>(vr + perm_row(2 * t) * 32 + 8 * 32);
    v[3] = *reinterpret_cast<const uint32_t *>(vr + perm_row(2 * t + 1) * 32 + 8 * 32);
  }

  // o += weights x values of plane p on integer products: the weights p s of a column as 16-bit
  // fixed-point numbers of their largest in the block, in two bytes (off by 2^-17 of the largest), codes as
  // they are.  The sums are exact; o holds channels 8g + 2 mt and 8g + 2 mt + 1.
  __device__ __forceinline__ void out_int(const uint8_t *blk, int p, int my_key, const float (*x)[4]) {
    float y[NSUP][4], t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int sp = 0; sp < NSUP; sp++) {
      const uint8_t *vp = blk + 2 * NG * PLANE + (NG + p) * PAIRS + (sp * NTI * 16 + my_key) * 4;
      const float2 s0 = pair_at(vp), s1 = pair_at(vp + 8 * 4);
      ofs[p][0] = fmaf(x[sp][0], s0.y, fmaf(x[sp][2], s1.y, ofs[p][0]));
      ofs[p][1] = fmaf(x[sp][1], s0.y, fmaf(x[sp][3], s1.y, ofs[p][1]));
      y[sp][0] = x[sp][0] * s0.x;
      y[sp][1] = x[sp][1] * s0.x;
      y[sp][2] = x[sp][2] * s1.x;
      y[sp][3] = x[sp][3] * s1.x;
      t0 = max3f(t0, y[sp][0], y[sp][2]);
      t1 = max3f(t1, y[sp][1], y[sp][3]);
    }
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, k));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, k));
    }
    t0 = fmaxf(t0, 0x1p-110f);  // the step stays a normal number
    t1 = fmaxf(t1, 0x1p-110f);
    const float i0 = __fdividef(65535.f, t0), i1 = __fdividef(65535.f, t1);
    uint32_t hb[4], lb[4];
    uint32_t lo[NSUP], hi[NSUP];  // bytes of column g's weights of the tile's rows 2t, 2t + 1, 8 + 2t, 8 + 2t + 1
#pragma unroll
    for (int sp = 0; sp < NSUP; sp++) {
      const uint32_t n0 = __float_as_uint(fmaf(y[sp][0], i0, MAGIC_F)), n1 = __float_as_uint(fmaf(y[sp][1], i1, MAGIC_F));
      const uint32_t n2 = __float_as_uint(fmaf(y[sp][2], i0, MAGIC_F)), n3 = __float_as_uint(fmaf(y[sp][3], i1, MAGIC_F));
      const uint32_t x0 = transpose8(__byte_perm(n0, n1, 0x5410)), x1 = transpose8(__byte_perm(n2, n3, 0x5410));
      lo[sp] = __byte_perm(x0, x1, 0x6420);
      hi[sp] = __byte_perm(x0, x1, 0x7531);
    }
    const int start[4] = {MAGIC, MAGIC, MAGIC, MAGIC};
    uint32_t vt[4][4];  // byte c of a tile's four keys: channels 8g + 2c (low) and 8g + 2c + 1 (high)
#pragma unroll
    for (int k = 0; k < 4; k++) {
      uint32_t v[4];
      v_words(blk, p, k, v);
      const uint32_t a01 = __byte_perm(v[0], v[1], 0x5140), b01 = __byte_perm(v[0], v[1], 0x7362);
      const uint32_t a23 = __byte_perm(v[2], v[3], 0x5140), b23 = __byte_perm(v[2], v[3], 0x7362);
      vt[k][0] = __byte_perm(a01, a23, 0x5410);
      vt[k][1] = __byte_perm(a01, a23, 0x7632);
      vt[k][2] = __byte_perm(b01, b23, 0x5410);
      vt[k][3] = __byte_perm(b01, b23, 0x7632);
      hb[k] = in_tile(hi[k / NTI], k % NTI);
      lb[k] = in_tile(lo[k / NTI], k % NTI);
    }
    const float e0 = t0 * (1.f / 65535.f), e1 = t1 * (1.f / 65535.f);
    const float e[4] = {e0, e1, e0 * 0.0625f, e1 * 0.0625f};
#pragma unroll
    for (int mt = 0; mt < 4; mt++) {
      int ah[4], al[4];
#pragma unroll
      for (int j = 0; j < 4; j += 2) {  // two 16-key tiles a product
        const uint32_t f[4] = {vt[j][mt] & 0x0f0f0f0fu, vt[j][mt] & 0xf0f0f0f0u, vt[j + 1][mt] & 0x0f0f0f0fu,
                               vt[j + 1][mt] & 0xf0f0f0f0u};  // odd channels: 16 c
        mma16832<false>(ah, f, hb[j], hb[j + 1], j == 0 ? start : ah);
        mma16832<false>(al, f, lb[j], lb[j + 1], j == 0 ? start : al);
      }
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const float v = fmaf(256.f, __int_as_float(ah[c]) - MAGIC_F, __int_as_float(al[c]) - MAGIC_F);
        o[p][mt][c] = fmaf(e[c], v, o[p][mt][c]);
      }
    }
  }

  // the same with float32 weights in three bf16 terms; o holds channels 8g + mt and 8g + 4 + mt
  __device__ __forceinline__ void out_float(const uint8_t *blk, int p, int my_key, const float (*x)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    float ob[4][4];  // the block's own sums, added in 32-bit rounding to nearest
#pragma unroll
    for (int mt = 0; mt < 4; mt++)
#pragma unroll
      for (int c = 0; c < 4; c++) ob[mt][c] = 0.f;
#pragma unroll
    for (int sp = 0; sp < NSUP; sp++) {
      const uint8_t *vp = blk + 2 * NG * PLANE + (NG + p) * PAIRS + (sp * NTI * 16 + my_key) * 4;
      const float2 s0 = pair_at(vp), s1 = pair_at(vp + 8 * 4);
      const float z0 = fmaf(8.f, s0.x, s0.y), z1 = fmaf(8.f, s1.x, s1.y);
      ofs[p][0] = fmaf(x[sp][0], z0, fmaf(x[sp][2], z1, ofs[p][0]));
      ofs[p][1] = fmaf(x[sp][1], z0, fmaf(x[sp][3], z1, ofs[p][1]));
      uint32_t bq[3][2];  // weights as B fragments: column g, keys perm(2t), perm(2t + 1) (+ 8)
      float y0 = x[sp][0] * s0.x, y1 = x[sp][1] * s0.x, y2 = x[sp][2] * s1.x, y3 = x[sp][3] * s1.x;
#pragma unroll
      for (int k = 0; k < 3; k++) {
        const uint32_t h0 = bf2_pack_rn(y0, y1), h1 = bf2_pack_rn(y2, y3);
        bq[k][0] = transpose8(h0);
        bq[k][1] = transpose8(h1);
        y0 -= __uint_as_float(h0 << 16);
        y1 -= __uint_as_float(h0 & 0xffff0000u);
        y2 -= __uint_as_float(h1 << 16);
        y3 -= __uint_as_float(h1 & 0xffff0000u);
      }
#pragma unroll
      for (int ti = 0; ti < NTI; ti++) {
        uint32_t v[4];
        v_words(blk, p, sp * NTI + ti, v);
        const uint32_t lo01 = __byte_perm(v[0], v[1], 0x5410), hi01 = __byte_perm(v[0], v[1], 0x7632);
        const uint32_t lo23 = __byte_perm(v[2], v[3], 0x5410), hi23 = __byte_perm(v[2], v[3], 0x7632);
        const bool on = GP == 8 || g / GP == ti;
        auto tile = [&](auto mtag) {
          constexpr int mt = decltype(mtag)::value;
          const uint32_t f[4] = {codes2<mt>(lo01), codes2<mt>(hi01), codes2<mt>(lo23), codes2<mt>(hi23)};
#pragma unroll
          for (int k = 2; k >= 0; k--) mma16816(ob[mt], f, on ? bq[k][0] : 0u, on ? bq[k][1] : 0u);
        };
        tile(std::integral_constant<int, 0>());
        tile(std::integral_constant<int, 1>());
        tile(std::integral_constant<int, 2>());
        tile(std::integral_constant<int, 3>());
      }
    }
#pragma unroll
    for (int mt = 0; mt < 4; mt++)
#pragma unroll
      for (int c = 0; c < 4; c++) o[p][mt][c] += ob[mt][c];
  }

  // Join the lanes' sums and the key tiles' columns: afterwards the lanes with 2 t < GP hold, for
  // the query heads 2 t and 2 t + 1, the maximum m2, the sum l2 and the outputs value(p, hf, mt, c).
  __device__ __forceinline__ void join() {
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
#pragma unroll
      for (int c = 0; c < 2; c++) {
        l2[c] += __shfl_xor_sync(0xffffffffu, l2[c], k);
#pragma unroll
        for (int p = 0; p < NG; p++) ofs[p][c] += __shfl_xor_sync(0xffffffffu, ofs[p][c], k);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; c++) {
      float m = m2[c];
#pragma unroll
      for (int k = GP / 2; k < 4; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      // a column with no key yet holds zeros (or what a NaN key left: kept)
      const float f = m2[c] == -INFINITY ? 1.f : tc::ex2(m2[c] - m);
      m2[c] = m;
      l2[c] *= f;
#pragma unroll
      for (int k = GP / 2; k < 4; k <<= 1) l2[c] += __shfl_xor_sync(0xffffffffu, l2[c], k);
#pragma unroll
      for (int p = 0; p < NG; p++)
#pragma unroll
        for (int mt = 0; mt < 4; mt++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            float v = (o[p][mt][c + 2 * hf] + ofs[p][c]) * f;
#pragma unroll
            for (int k = GP / 2; k < 4; k <<= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
            o[p][mt][c + 2 * hf] = v;
          }
    }
  }
  // four consecutive channels p * 64 + 8 g + 4 hf .. of query head 2 t + c (after join)
  __device__ __forceinline__ float4 value(int p, int hf, int c) const {
    if constexpr (INT)
      return make_float4(o[p][2 * hf][c], o[p][2 * hf][c + 2], o[p][2 * hf + 1][c], o[p][2 * hf + 1][c + 2]);
    return make_float4(o[p][0][c + 2 * hf], o[p][1][c + 2 * hf], o[p][2][c + 2 * hf], o[p][3][c + 2 * hf]);
  }
};

// Ring of a warp's blocks in shared memory.  wait() answers the same in every lane: what follows it is
// done by whole warps, and at the limit the lanes' own answers may differ (one more look each).
template <int BLK, int ST>
struct Ring {
  uint8_t *mem;
  uint64_t *bars;
  volatile int *abort;
  int *err;
#ifdef DREAMER_TEST_HOOKS
  int withhold = -1;  // this copy is announced and never made
#endif
  __device__ __forceinline__ void issue(uint32_t i, const uint8_t *src) const {
    const uint32_t bar = tc::smem_u32(&bars[i % ST]);
    tc::mbar_expect_tx(bar, BLK);
#ifdef DREAMER_TEST_HOOKS
    if ((int)i == withhold) return;
#endif
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(mem + (i % ST) * BLK)),
        "l"(src), "r"((uint32_t)BLK), "r"(bar)
        : "memory");
  }
  __device__ __forceinline__ bool wait(uint32_t i) const {
    return __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&bars[i % ST]), (i / ST) & 1, abort, err));
  }
  // after an expired wait: the copies i0 .. i1 - 1, still in flight, land (or time out) before the exit
  __device__ __forceinline__ void drain(uint32_t i0, uint32_t i1) const {
    for (uint32_t i = i0; i < i1; i++) {
      const uint64_t t0 = tc::globaltimer();
      while (!tc::mbar_try_wait(tc::smem_u32(&bars[i % ST]), (i / ST) & 1) &&
             tc::globaltimer() - t0 < tc::WAIT_LIMIT_NS) {
      }
    }
  }
};

// Keys of sequence b; a length outside 0 .. limit is reported and counts as none
__device__ __forceinline__ int keys_of(const AttnArgs &a, int b, bool report) {
  const long len = (long)a.lens[b] + a.len_add;
  if (len < 0 || len > a.limit) {
    if (report) raise_dev_error(a.err, DEV_BAD_INDEX);
    return 0;
  }
  return (int)len;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

// Cluster form (one launch): a cluster of CTAs takes one (sequence, key head, chunk of GP
// query heads), every CTA a contiguous share of its blocks, every warp each NW-th block of that;
// warps join in shared memory, CTAs in distributed shared memory.
template <typename T, int NG, int GP, int NW, int ST, int OCC>
__global__ void __launch_bounds__(NW * 32, OCC) kv4_attn_kernel(AttnArgs a) {
  using W = WarpAttn<T, NG, GP>;
  constexpr int D = W::D, BLK = W::BLK;
  extern __shared__ __align__(128) uint8_t ring_mem[];  // rings; then [NW][GP][D] partial outputs
  __shared__ __align__(8) uint64_t bars[NW * ST];
  __shared__ float sm_m[NW][GP], sm_l[NW][GP];
  __shared__ float so[GP][D], sM[GP], sL[GP];
  __shared__ int s_abort;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint32_t crank, csize;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int item = blockIdx.x / csize;
  const int qc = item % a.qchunks, pair = item / a.qchunks;
  const int b = pair / a.Hkv, kvh = pair % a.Hkv;
  const int nq = min(GP, a.G - qc * GP);
  const int head0 = kvh * a.G + qc * GP;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NW * ST; i++) tc::mbar_init(tc::smem_u32(&bars[i]), 1);
    tc::fence_mbar_init();
    s_abort = 0;
  }
  __syncthreads();
  const int nkeys = keys_of(a, b, threadIdx.x == 0);
  const int nb = (nkeys + KV4_BLOCK - 1) / KV4_BLOCK;
  const int per = (nb + (int)csize - 1) / (int)csize;
  const int blk0 = min(nb, (int)crank * per), blk1 = min(nb, blk0 + per);
  const uint8_t *base = a.data + (long)pair * (a.cap / KV4_BLOCK) * BLK;
  const int mine = blk1 - blk0 > warp ? (blk1 - blk0 - warp + NW - 1) / NW : 0;
  Ring<BLK, ST> ring{ring_mem + warp * ST * BLK, bars + warp * ST, &s_abort, a.err};
#ifdef DREAMER_TEST_HOOKS
  ring.withhold = a.withhold.copy_of(blockIdx.x, warp);
#endif
  auto src = [&](int i) { return base + (long)(blk0 + warp + i * NW) * BLK; };
  if (lane == 0)
    for (int i = 0; i < ST && i < mine; i++) ring.issue(i, src(i));
  W w;
  w.start(reinterpret_cast<const T *>(a.q) + (long)b * a.ldq + (long)head0 * D, nq, a.scale_log2);
  bool expired = false;
  for (int i = 0; i < mine; i++) {
    if (!ring.wait(i)) {
      if (lane == 0) ring.drain(i, min(mine, i + ST));
      expired = true;
      break;
    }
    w.block(ring.mem + (i % ST) * BLK, (blk0 + warp + i * NW) * KV4_BLOCK, nkeys);
    __syncwarp();
    if (lane == 0 && i + ST < mine) ring.issue(i + ST, src(i + ST));  // into the stage just read
  }
  w.join();
  if (expired) w.l2[0] = w.l2[1] = NAN;  // the item's sum, and so its output in every CTA of the cluster
  __syncthreads();  // every warp is done with the rings
  float *part = reinterpret_cast<float *>(ring_mem);
  if (2 * t < GP) {
#pragma unroll
    for (int c = 0; c < 2; c++) {
      const int qh = 2 * t + c;
      if (g == 0) {
        sm_m[warp][qh] = w.m2[c];
        sm_l[warp][qh] = w.l2[c];
      }
#pragma unroll
      for (int p = 0; p < NG; p++)
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
          *reinterpret_cast<float4 *>(part + (warp * GP + qh) * D + p * 64 + 8 * g + 4 * hf) = w.value(p, hf, c);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < GP * D; e += NW * 32) {
    const int qh = e / D;
    float m = sm_m[0][qh];
#pragma unroll
    for (int k = 1; k < NW; k++) m = fmaxf(m, sm_m[k][qh]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int k = 0; k < NW; k++) {
      const float f = sm_m[k][qh] == -INFINITY ? 1.f : tc::ex2(sm_m[k][qh] - m);
      acc = fmaf(f, part[k * GP * D + e], acc);
      l = fmaf(f, sm_l[k][qh], l);
    }
    so[qh][e % D] = acc;
    if (e % D == 0) {
      sM[qh] = m;
      sL[qh] = l;
    }
  }
  // every CTA of the cluster writes its share of the output
  if (csize > 1) cluster_sync();
  else __syncthreads();
  for (int e = (int)crank * (NW * 32) + threadIdx.x; e < nq * D; e += (int)csize * (NW * 32)) {
    const int qh = e / D;
    float acc = 0.f, l = 0.f;
    if (csize > 1) {
      float m = -INFINITY;
      const uint32_t aM = tc::smem_u32(&sM[qh]), aL = tc::smem_u32(&sL[qh]), aO = tc::smem_u32(&so[qh][e % D]);
      for (uint32_t r = 0; r < csize; r++) m = fmaxf(m, ld_cluster(map_to_rank(aM, r)));
      for (uint32_t r = 0; r < csize; r++) {
        const float mr = ld_cluster(map_to_rank(aM, r));
        const float f = mr == -INFINITY ? 1.f : tc::ex2(mr - m);
        acc = fmaf(f, ld_cluster(map_to_rank(aO, r)), acc);
        l = fmaf(f, ld_cluster(map_to_rank(aL, r)), l);
      }
    } else {
      acc = so[qh][e % D];
      l = sL[qh];
    }
    const float res = nkeys == 0 ? 0.f : acc / l;
    reinterpret_cast<T *>(a.out)[(long)b * a.ldo + (long)(head0 + qh) * D + e % D] = from_f<T>(res);
  }
  if (csize > 1) cluster_sync();  // shared memory that others read stays until they have
}

// Split form: the blocks of all items (sequence, key head, chunk of query heads) form one
// sequence, item by item, and every warp of a grid that fills the GPU once takes an equal run of it,
// whatever the lengths.  A warp that holds a whole item writes its output; the others leave
// partial outputs in slot (warp + item), and kv4_join_kernel joins an item's slots, which are
// consecutive.  Where all of a CTA's runs lie in one item, its warps join first and leave one slot,
// that of the first warp.
__device__ __forceinline__ int warp_incl_sum(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += u;
  }
  return v;
}
// Starting and ending an item costs a warp about as much as ITEM_COST blocks (q, the joins): an item
// of n blocks counts as n + ITEM_COST, its blocks being the last n.
constexpr int ITEM_COST = 2;
__device__ __forceinline__ int blocks_of(const AttnArgs &a, int b) {
  return (keys_of(a, b, false) + KV4_BLOCK - 1) / KV4_BLOCK;
}
__device__ __forceinline__ int cost_of(int blocks) { return blocks > 0 ? blocks + ITEM_COST : 0; }

template <typename T, int NG, int GP, int NW, int ST, int OCC>
__global__ void __launch_bounds__(NW * 32, OCC) kv4_split_kernel(AttnArgs a) {
  using W = WarpAttn<T, NG, GP>;
  constexpr int D = W::D, BLK = W::BLK;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ __align__(8) uint64_t bars[NW * ST];
  __shared__ int s_abort;
  __shared__ int s_one;  // item + 1 where the CTA's runs lie in one item and leave one slot, else 0
  __shared__ float sm_m[NW][GP], sm_l[NW][GP];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NW * ST; i++) tc::mbar_init(tc::smem_u32(&bars[i]), 1);
    tc::fence_mbar_init();
    s_abort = 0;
    s_one = 0;
  }
  if (blockIdx.x == 0 && warp == 0)
    for (int i = lane; i < a.B; i += 32) keys_of(a, i, true);
  __syncthreads();
  const int gw = blockIdx.x * NW + warp;
  const int per_seq = a.Hkv * a.qchunks;
  int total = 0;
  for (int i = lane; i < a.B; i += 32) total += cost_of(blocks_of(a, i));
  total = __reduce_add_sync(0xffffffffu, total) * per_seq;
  const int per = (total + a.n_warps - 1) / a.n_warps;
  const int f0 = min((long)gw * per, (long)total), f1 = min((long)f0 + per, (long)total);
  const long c0 = (long)blockIdx.x * NW * per, c1 = min(c0 + (long)NW * per, (long)total);  // of the CTA
  if (c0 >= c1) return;  // the whole CTA
  bool one = false;
  if (f0 < f1) {
  // the sequence that f0 lies in, and the cost before it
  int b = 0, before = 0;
  for (int i0 = 0, sum = 0; i0 < a.B; i0 += 32) {
    const int n = i0 + lane < a.B ? cost_of(blocks_of(a, i0 + lane)) * per_seq : 0;
    const int incl = sum + warp_incl_sum(n);
    const unsigned past = __ballot_sync(0xffffffffu, incl > f0);
    if (past) {
      const int k = __ffs(past) - 1;
      b = i0 + k;
      before = __shfl_sync(0xffffffffu, incl - n, k);
      break;
    }
    sum = __shfl_sync(0xffffffffu, incl, 31);
  }
  // the run, walked twice: by the issue of copies (ld_) and, up to ST blocks behind it, by the
  // arithmetic; `v` is the place of the next block in the sequence of costs
  const int cap_blk = a.cap / KV4_BLOCK;
  auto next_blocks = [&](int &sq) {  // blocks of the first sequence from sq on that has a key
    for (;; sq++) {
      const int nb = blocks_of(a, sq);
      if (nb > 0) return nb;
    }
  };
  int nb = blocks_of(a, b);
  int it = (f0 - before) / cost_of(nb);
  const int first = before + it * cost_of(nb) + ITEM_COST;  // place of the item's block 0
  int v = max(f0, first), blk = v - first;
  one = first <= c0 && c1 <= first + nb && per < nb;
  Ring<BLK, ST> ring{ring_mem + warp * ST * BLK, bars + warp * ST, &s_abort, a.err};
#ifdef DREAMER_TEST_HOOKS
  ring.withhold = a.withhold.copy_of(blockIdx.x, warp);
#endif
  int issued = 0, ld_v = v, ld_b = b, ld_it = it, ld_nb = nb, ld_left = nb - blk;
  const uint8_t *ld = a.data + ((long)(b * a.Hkv + it / a.qchunks) * cap_blk + blk) * BLK;
  auto issue_next = [&]() {
    if (lane == 0) ring.issue(issued, ld);
    issued++;
    ld_v++;
    ld += BLK;
    if (--ld_left == 0 && ld_v < f1) {  // the next item
      ld_v += ITEM_COST;
      if (++ld_it == per_seq) {
        ld_it = 0;
        ld_b++;
        ld_nb = next_blocks(ld_b);
      }
      ld_left = ld_nb;
      ld = a.data + (long)(ld_b * a.Hkv + ld_it / a.qchunks) * cap_blk * BLK;
    }
  };
  for (int i = 0; i < ST && ld_v < f1; i++) issue_next();
  W w;
  bool expired = false;  // a wait was: this and the run's further items become NaN
  for (int i = 0; v < f1;) {  // segments of one item each
    const int kvh = it / a.qchunks, qc = it % a.qchunks;
    const int head0 = kvh * a.G + qc * GP, nq = min(GP, a.G - qc * GP);
    const int nkeys = keys_of(a, b, false);
    const int take = min(nb - blk, f1 - v);
    w.start(reinterpret_cast<const T *>(a.q) + (long)b * a.ldq + (long)head0 * D, nq, a.scale_log2);
    for (int k = 0; k < take && !expired; k++, i++) {
      if (!ring.wait(i)) {
        if (lane == 0) ring.drain(i, issued);
        expired = true;
        break;
      }
      w.block(ring.mem + (i % ST) * BLK, (blk + k) * KV4_BLOCK, nkeys);
      __syncwarp();
      if (ld_v < f1) issue_next();  // into the stage just read
    }
    w.join();
    if (expired) w.l2[0] = w.l2[1] = NAN;
    if (2 * t < GP) {
      if (one) {  // into the warp's own stages, all read
        float *dst = reinterpret_cast<float *>(ring.mem);
#pragma unroll
        for (int k = 0; k < 2; k++) {
          if (g == 0) {
            sm_m[warp][2 * t + k] = w.m2[k];
            sm_l[warp][2 * t + k] = w.l2[k];
          }
#pragma unroll
          for (int p = 0; p < NG; p++)
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
              *reinterpret_cast<float4 *>(dst + (2 * t + k) * D + p * 64 + 8 * g + 4 * hf) = w.value(p, hf, k);
        }
        if (warp == 0 && lane == 0) s_one = b * per_seq + it + 1;
      } else if (take == nb) {
        T *dst = reinterpret_cast<T *>(a.out) + (long)b * a.ldo + (long)head0 * D;
#pragma unroll
        for (int k = 0; k < 2; k++)
          if (2 * t + k < nq) {
            const float inv = 1.f / w.l2[k];
#pragma unroll
            for (int p = 0; p < NG; p++) {
              const float4 u = w.value(p, 0, k), v = w.value(p, 1, k);
              const float r[8] = {u.x * inv, u.y * inv, u.z * inv, u.w * inv, v.x * inv, v.y * inv, v.z * inv, v.w * inv};
              store8(dst + (2 * t + k) * D + p * 64 + 8 * g, r);
            }
          }
      } else {
        float *dst = a.part + (long)(gw + b * per_seq + it) * GP * (D + 4);
#pragma unroll
        for (int k = 0; k < 2; k++)
          if (2 * t + k < nq) {
            float *d = dst + (2 * t + k) * (D + 4);
#pragma unroll
            for (int p = 0; p < NG; p++)
#pragma unroll
              for (int hf = 0; hf < 2; hf++)
                *reinterpret_cast<float4 *>(d + p * 64 + 8 * g + 4 * hf) = w.value(p, hf, k);
            if (g == 0) *reinterpret_cast<float2 *>(d + D) = make_float2(w.m2[k], w.l2[k]);
          }
      }
    }
    v += take;
    if (v < f1) {  // the next item
      v += ITEM_COST;
      blk = 0;
      if (++it == per_seq) {
        it = 0;
        b++;
        nb = next_blocks(b);
      }
    }
  }
  } else if (warp > 0 && lane < GP) {  // no blocks: nothing to add to the CTA's item
    sm_m[warp][lane] = -INFINITY;
    sm_l[warp][lane] = 0.f;
  }
  __syncthreads();
  if (s_one == 0) return;
  // one slot of the CTA
  float *dst = a.part + (long)(blockIdx.x * NW + s_one - 1) * GP * (D + 4);
  static_assert(GP * D * 4 <= ST * BLK, "a warp's stages hold its partial output");
  for (int e = threadIdx.x; e < GP * D; e += NW * 32) {
    const int qh = e / D;
    float m = sm_m[0][qh];
#pragma unroll
    for (int k = 1; k < NW; k++) m = fmaxf(m, sm_m[k][qh]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int k = 0; k < NW; k++) {
      const bool none = c0 + k * (long)per >= c1;  // a warp without blocks
      const float f = none ? 0.f : sm_m[k][qh] == -INFINITY ? 1.f : tc::ex2(sm_m[k][qh] - m);
      if (!none) acc = fmaf(f, reinterpret_cast<const float *>(ring_mem + k * ST * BLK)[e], acc);
      l = fmaf(f, sm_l[k][qh], l);
    }
    dst[qh * (D + 4) + e % D] = acc;
    if (e % D == 0) *reinterpret_cast<float2 *>(dst + qh * (D + 4) + D) = make_float2(m, l);
  }
}

// Join the slots of an item's query head: `share` warps of a CTA (1 to 8) take turns at its slots, a
// lane D / 32 channels, then join in shared memory.  An item's slots are those of the warps that hold a
// part of it, one a CTA where the whole CTA does.  Items that one warp held are done; items without a
// key get zeros.
template <typename T, int D, int GP, int SNW>
__global__ void __launch_bounds__(256) kv4_join_kernel(AttnArgs a, int share) {
  constexpr int NW = 8, C = D / 32;
  __shared__ float so[NW][D], sm[NW], sl[NW];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = a.Hkv * a.qchunks, Hq = a.Hkv * a.G;
  const int part_of = warp % share;  // this warp's turn
  const long out = (long)blockIdx.x * (NW / share) + warp / share;
  const bool live = out < (long)a.B * Hq;
  const int b = live ? (int)(out / Hq) : 0, head = live ? (int)(out % Hq) : 0;
  const int kvh = head / a.G, qh = head % a.G;
  const int it = kvh * a.qchunks + qh / GP;
  int sum = 0, upto = 0;  // cost of all sequences, and of those before b
  for (int i = lane; i < a.B; i += 32) {
    const int n = cost_of(blocks_of(a, i));
    sum += n;
    upto += i < b ? n : 0;
  }
  sum = __reduce_add_sync(0xffffffffu, sum) * per_seq;
  upto = __reduce_add_sync(0xffffffffu, upto) * per_seq;
  const int nb = blocks_of(a, b);
  const int per = (sum + a.n_warps - 1) / a.n_warps;
  const int s = upto + it * cost_of(nb) + ITEM_COST;  // places of the blocks: s .. s + nb - 1
  const int w0 = nb ? s / per : 0, w1 = nb ? (s + nb - 1) / per : 0;
  float m = -INFINITY, l = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; c++) acc[c] = 0.f;
  const bool held = w0 == w1;  // by one warp (or no block at all)
  if (live && !held) {
    // the CTAs cA .. cB hold the item: one slot each, but the first and the last a slot a warp where
    // they hold another item too
    auto joined = [&](int c) {  // as in the split kernel
      const long c0 = (long)c * SNW * per, c1 = min(c0 + (long)SNW * per, (long)sum);
      return s <= c0 && c1 <= s + nb && per < nb;
    };
    const int cA = w0 / SNW, cB = w1 / SNW;
    const int nA = joined(cA) ? 1 : min(w1, cA * SNW + SNW - 1) - w0 + 1;
    const int mid = max(0, cB - cA - 1);
    const int nB = cA == cB ? 0 : joined(cB) ? 1 : w1 - cB * SNW + 1;
    const int n = nA + mid + nB;
    const long step = (long)GP * (D + 4);
    const float *base = a.part + ((long)(b * per_seq + it) * GP + qh % GP) * (D + 4);
    auto slot = [&](int j) {
      const int w = j < nA ? w0 + j : j < nA + mid ? (cA + 1 + j - nA) * SNW : cB * SNW + j - nA - mid;
      return base + w * step;
    };
    // eight slots a step, their loads in flight together
    for (int i = part_of; i < n; i += 8 * share) {
      float2 ml[8];
      float v[8][C];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const int j = i + k * share;
        ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int c = 0; c < C; c++) v[k][c] = 0.f;
        if (j < n) {
          const float *p = slot(j);
          ml[k] = *reinterpret_cast<const float2 *>(p + D);
          if constexpr (C == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + 4 * lane);
            v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2 *>(p + 2 * lane);
            v[k][0] = x.x; v[k][1] = x.y;
          }
        }
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < 8; k++) mn = fmaxf(mn, ml[k].x);
      const float al = m == -INFINITY ? 1.f : tc::ex2(m - mn);
      l *= al;
#pragma unroll
      for (int c = 0; c < C; c++) acc[c] *= al;
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float f = ml[k].x == -INFINITY ? 1.f : tc::ex2(ml[k].x - mn);
        l = fmaf(f, ml[k].y, l);
#pragma unroll
        for (int c = 0; c < C; c++) acc[c] = fmaf(f, v[k][c], acc[c]);
      }
      m = mn;
    }
  }
  if (share > 1) {
#pragma unroll
    for (int c = 0; c < C; c++) so[warp][C * lane + c] = acc[c];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    if (part_of) return;
    for (int k = warp + 1; k < warp + share; k++) {
      const float mn = fmaxf(m, sm[k]);
      const float f0 = m == -INFINITY ? 1.f : tc::ex2(m - mn), f1 = sm[k] == -INFINITY ? 1.f : tc::ex2(sm[k] - mn);
      l = fmaf(f1, sl[k], l * f0);
#pragma unroll
      for (int c = 0; c < C; c++) acc[c] = fmaf(f1, so[k][C * lane + c], acc[c] * f0);
      m = mn;
    }
  }
  if (!live || (held && nb)) return;
  T *dst = reinterpret_cast<T *>(a.out) + (long)b * a.ldo + (long)head * D;
  const float inv = nb ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < C; c++) dst[C * lane + c] = from_f<T>(nb ? acc[c] * inv : 0.f);
}

RowArgs row_args(const Kv4Cache &c, const Kv4Rows &r) {
  RowArgs a{};
  a.data = c.data;
  a.B = c.B; a.Hkv = c.Hkv; a.ng = c.d / KV4_GROUP; a.cap = c.cap;
  a.k = r.k; a.v = r.v; a.ldk = r.ldk; a.ldv = r.ldv;
  a.cu = r.cu; a.start = r.start; a.n_rows = r.n_rows; a.zero_rest = r.zero_rest; a.err = r.err;
  a.limit = r.limit ? r.limit : c.cap;
  return a;
}
dim3 row_grid(const RowArgs &a, int rows) {
  return dim3((a.n_rows + rows - 1) / rows, (a.Hkv * a.ng + 7) / 8, 2);
}
int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return 148;
  return sms;
}

// 64 rows a CTA from two CTAs an SM on
bool many_rows(const RowArgs &a) {
  const dim3 g = row_grid(a, 64);
  return (long)g.x * g.y * g.z >= 2L * device_sms();
}

// Warps a CTA, ring stages and CTAs an SM (a third stage, or a fifth CTA, measured no faster)
template <typename T, int NG> struct FormCfg {
  static constexpr int NW = 4;
  static constexpr int ST = NG == 1 ? 3 : 2;
  static constexpr int OCC = sizeof(T) == 4 ? 2 : NG == 1 ? 4 : 3;
};

int heads_a_chunk(int G) { return G <= 2 ? 2 : G <= 4 ? 4 : 8; }

// How the items are spread over the GPU's `slots` CTAs, from the number of items and the most blocks
// of one (the lengths are known on the device only).  A cluster form's CTAs join by themselves, the
// hardware hands out what does not fit at once, and equal lengths keep every warp busy.  The split form
// pays a second launch and evens out what a single wave cannot.  Its time against the cluster form's, both
// forced, bfloat16, 4 to 512 items of one head of 64 and of four of 128, all of the full length | ragged:
//   clusters of 8:      4 blocks a warp -2 .. +25 % | -3 .. +15;   6: -18 .. +17 | -17 .. +8;   16: -41 .. +8 | -42 .. -14
//   of 4, 2, no others: 8 blocks a warp +15 .. +23 % | -8 .. +15;  12: +9 .. +16 | -28 .. +10;  16: +7 .. +13 | -26 .. -2;
//                       32 to 128: -9 .. -1 | -54 .. -14
// so from 6 and 12 blocks on the split form is taken, for lengths that differ: 128 items of up to 12288 tokens 45 ->
// 24 us, all of 12288 51 -> 50; 4 of 32768 26 -> 15.
struct Plan {
  int cluster;
  bool split;
};
Plan plan_for(long items, int nblk, long slots, int nw) {
  Plan p{1, false};
  while (p.cluster < 8 && items * p.cluster * 2 <= slots && nblk > nw * p.cluster) p.cluster *= 2;
  p.split = items * p.cluster <= slots && nblk >= nw * p.cluster * (p.cluster == 8 ? 6 : 12);
  return p;
}

template <typename T, int NG, int GP>
int launch_attn(AttnArgs a, cudaStream_t s, LaunchOpt o) {
  using W = WarpAttn<T, NG, GP>;
  a.qchunks = (a.G + GP - 1) / GP;
  const long items = (long)a.B * a.Hkv * a.qchunks;
  const int nblk = a.cap / KV4_BLOCK;
  if (items * (nblk + ITEM_COST) >= 0x7fffffffL) return DREAMER_ERR_UNSUPPORTED;
  using C = FormCfg<T, NG>;
  const int sms = device_sms();
  const Plan p = plan_for(items, nblk, (long)sms * C::OCC, C::NW);
  if (p.split) {
    const int grid = sms * C::OCC;
    a.n_warps = grid * C::NW;
    const int rc = launch<kv4_split_kernel<T, NG, GP, C::NW, C::ST, C::OCC>>(dim3(grid), dim3(C::NW * 32),
                                                                             C::NW * C::ST * W::BLK, 1, s, o, a);
    if (rc) return rc;
    LaunchOpt j;
    j.pdl = o.next;  // the split kernel precedes it on the stream
    // warps a query head: one for each four of the slots that items have on average
    const long outs = (long)a.B * a.Hkv * a.G, mean = a.n_warps / items;
    const int share = mean > 64 ? 8 : mean > 32 ? 4 : mean > 8 ? 2 : 1;
    return launch<kv4_join_kernel<T, W::D, GP, C::NW>>(dim3((unsigned)((outs * share + 7) / 8)), dim3(256), 0, 1, s, j, a,
                                                       share);
  }
  constexpr int part = C::NW * GP * W::D * 4, rings = C::NW * C::ST * W::BLK;
  return launch<kv4_attn_kernel<T, NG, GP, C::NW, C::ST, C::OCC>>(dim3((unsigned)(items * p.cluster)), dim3(C::NW * 32),
                                                          rings > part ? rings : part, p.cluster, s, o, a);
}

template <typename T, int NG>
int dispatch_attn(const AttnArgs &a, cudaStream_t s, LaunchOpt o) {
  switch (heads_a_chunk(a.G)) {
    case 2: return launch_attn<T, NG, 2>(a, s, o);
    case 4: return launch_attn<T, NG, 4>(a, s, o);
    default: return launch_attn<T, NG, 8>(a, s, o);
  }
}

}  // namespace

int kv4_store(const Kv4Cache &c, const Kv4Rows &r, cudaStream_t s, LaunchOpt o) {
  if (r.n_rows == 0) return DREAMER_OK;
  const RowArgs a = row_args(c, r);
  const bool f32 = r.dtype == 0;
  if (many_rows(a)) {
    const dim3 g = row_grid(a, 64);
    return f32 ? launch<kv4_store_kernel<float, 64>>(g, dim3(256), 0, 1, s, o, a)
               : launch<kv4_store_kernel<bf16, 64>>(g, dim3(256), 0, 1, s, o, a);
  }
  const dim3 g = row_grid(a, 16);
  return f32 ? launch<kv4_store_kernel<float, 16>>(g, dim3(256), 0, 1, s, o, a)
             : launch<kv4_store_kernel<bf16, 16>>(g, dim3(256), 0, 1, s, o, a);
}

int kv4_load(const Kv4Cache &c, const Kv4Rows &r, cudaStream_t s, LaunchOpt o) {
  if (r.n_rows == 0) return DREAMER_OK;
  const RowArgs a = row_args(c, r);
  const bool f32 = r.dtype == 0;
  if (many_rows(a)) {
    const dim3 g = row_grid(a, 64);
    return f32 ? launch<kv4_load_kernel<float, 64>>(g, dim3(256), 0, 1, s, o, a)
               : launch<kv4_load_kernel<bf16, 64>>(g, dim3(256), 0, 1, s, o, a);
  }
  const dim3 g = row_grid(a, 16);
  return f32 ? launch<kv4_load_kernel<float, 16>>(g, dim3(256), 0, 1, s, o, a)
             : launch<kv4_load_kernel<bf16, 16>>(g, dim3(256), 0, 1, s, o, a);
}

int kv4_attn(const Kv4Cache &c, const Kv4Attn &t, cudaStream_t s, LaunchOpt o) {
  AttnArgs a{};
  a.data = c.data;
  a.B = c.B; a.Hkv = c.Hkv; a.cap = c.cap; a.Hq = t.Hq; a.G = t.Hq / c.Hkv;
  a.q = t.q; a.ldq = t.ldq; a.out = t.out; a.ldo = t.ldo;
  a.lens = t.lens; a.len_add = t.len_add;
  a.limit = t.limit ? t.limit : c.cap;
  a.scale_log2 = t.scale * LOG2_E;
  a.err = t.err;
  a.part = (float *)t.workspace;
#ifdef DREAMER_TEST_HOOKS
  a.withhold = take_withhold();
#endif
  if (c.d == 64) return t.dtype == 0 ? dispatch_attn<float, 1>(a, s, o) : dispatch_attn<bf16, 1>(a, s, o);
  return t.dtype == 0 ? dispatch_attn<float, 2>(a, s, o) : dispatch_attn<bf16, 2>(a, s, o);
}

int kv4_attn_launches(const Kv4Cache &c, int Hq, int dtype) {
  const int G = Hq / c.Hkv, gp = heads_a_chunk(G);
  const long items = (long)c.B * c.Hkv * ((G + gp - 1) / gp);
  const int occ = dtype == 0 ? FormCfg<float, 1>::OCC : c.d == 64 ? FormCfg<bf16, 1>::OCC : FormCfg<bf16, 2>::OCC;
  return plan_for(items, c.cap / KV4_BLOCK, (long)device_sms() * occ, 4).split ? 2 : 1;
}

long kv4_attn_workspace(const Kv4Cache &c, int Hq, bool any_capacity) {
  const int G = Hq / c.Hkv, gp = heads_a_chunk(G);
  const long items = (long)c.B * c.Hkv * ((G + gp - 1) / gp);
  const int nblk = c.cap / KV4_BLOCK, sms = device_sms();
  const int occ = c.d == 64 ? FormCfg<bf16, 1>::OCC : FormCfg<bf16, 2>::OCC;
  if (!any_capacity && !plan_for(items, nblk, (long)sms * occ, 4).split &&
      !plan_for(items, nblk, (long)sms * FormCfg<float, 1>::OCC, 4).split)
    return 0;
  const long warps = (long)sms * 16;  // of either type
  return (warps + items) * gp * (c.d + 4) * (long)sizeof(float);
}

}  // namespace ops
}  // namespace dreamer

// ---- C entry points ----------------------------------------------------------------------
using namespace dreamer;

static bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

static int check_cache(const dreamer_kv4_cache *c) {
  if (!c || !c->data || !al16(c->data)) return DREAMER_ERR_ARG;
  if (c->batch < 1 || c->n_kv_heads < 1 || c->head_dim < 1 || c->capacity < 1) return DREAMER_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return DREAMER_ERR_UNSUPPORTED;
  if (c->capacity % ops::KV4_BLOCK) return DREAMER_ERR_UNSUPPORTED;
  if ((long)c->batch * c->n_kv_heads > (1L << 24)) return DREAMER_ERR_UNSUPPORTED;
  return DREAMER_OK;
}
static ops::Kv4Cache to_cache(const dreamer_kv4_cache *c) {
  return ops::Kv4Cache{(uint8_t *)c->data, c->batch, c->n_kv_heads, c->head_dim, c->capacity};
}

extern "C" int64_t dreamer_kv4_bytes(int batch, int n_kv_heads, int head_dim, int capacity) {
  if (batch < 1 || n_kv_heads < 1 || capacity < 1 || (head_dim != 64 && head_dim != 128) ||
      capacity % ops::KV4_BLOCK)
    return 0;
  return (int64_t)batch * n_kv_heads * (capacity / ops::KV4_BLOCK) * ops::kv4_block_bytes(head_dim);
}

static int check_rows(const dreamer_kv4_cache *c, const void *k, int64_t ldk, const void *v, int64_t ldv,
                      const int32_t *cu_rows, const int32_t *start, int n_rows, int dtype) {
  const int rc = check_cache(c);
  if (rc) return rc;
  if (!k || !v || !cu_rows || !start || n_rows < 0 || (dtype != 0 && dtype != 1)) return DREAMER_ERR_ARG;
  const int es = dtype == 0 ? 4 : 2;
  const int64_t w = (int64_t)c->n_kv_heads * c->head_dim;
  if (!al16(k) || !al16(v) || ldk < w || ldv < w || (ldk * es) % 16 || (ldv * es) % 16) return DREAMER_ERR_ARG;
  if ((long)c->n_kv_heads * c->head_dim > 64L * 8 * 65535) return DREAMER_ERR_UNSUPPORTED;
  return DREAMER_OK;
}

extern "C" int dreamer_kv4_store(const dreamer_kv4_cache *c, const void *k, int64_t ldk, const void *v,
                                 int64_t ldv, const int32_t *cu_rows, const int32_t *start, int n_rows,
                                 int dtype, int32_t *status, dreamer_stream stream) {
  const int rc = check_rows(c, k, ldk, v, ldv, cu_rows, start, n_rows, dtype);
  if (rc) return rc;
  return ops::kv4_store(to_cache(c), ops::Kv4Rows{k, v, ldk, ldv, cu_rows, start, n_rows, dtype, 0, status, 0},
                        (cudaStream_t)stream, ops::user_launch((cudaStream_t)stream));
}

extern "C" int dreamer_kv4_load(const dreamer_kv4_cache *c, void *k, int64_t ldk, void *v, int64_t ldv,
                                const int32_t *cu_rows, const int32_t *start, int n_rows, int dtype,
                                int zero_rest, int32_t *status, dreamer_stream stream) {
  const int rc = check_rows(c, k, ldk, v, ldv, cu_rows, start, n_rows, dtype);
  if (rc) return rc;
  return ops::kv4_load(to_cache(c), ops::Kv4Rows{k, v, ldk, ldv, cu_rows, start, n_rows, dtype, zero_rest ? 1 : 0, status, 0},
                       (cudaStream_t)stream, ops::user_launch((cudaStream_t)stream));
}

extern "C" int64_t dreamer_attn_kv4_workspace(const dreamer_kv4_cache *c, int n_heads) {
  if (!c || c->batch < 1 || c->n_kv_heads < 1 || n_heads < 1 || n_heads % c->n_kv_heads ||
      !dreamer_kv4_bytes(c->batch, c->n_kv_heads, c->head_dim, c->capacity))
    return 0;
  return ops::kv4_attn_workspace(to_cache(c), n_heads);
}

extern "C" int dreamer_attn_kv4(const dreamer_kv4_cache *c, const void *q, int64_t ldq, void *out, int64_t ldo,
                                const int32_t *lens, int n_heads, int dtype, float scale, void *workspace,
                                int64_t workspace_bytes, int32_t *status, dreamer_stream stream) {
  const int rc = check_cache(c);
  if (rc) return rc;
  if (!q || !out || !lens || n_heads < 1 || n_heads % c->n_kv_heads || (dtype != 0 && dtype != 1) ||
      !ops::scale_ok(scale))
    return DREAMER_ERR_ARG;
  const int es = dtype == 0 ? 4 : 2;
  const int64_t w = (int64_t)n_heads * c->head_dim;
  if (!al16(q) || !al16(out) || ldq < w || ldo < w || (ldq * es) % 16 || (ldo * es) % 16) return DREAMER_ERR_ARG;
  const int64_t need = ops::kv4_attn_workspace(to_cache(c), n_heads);
  if (need > 0 && (!workspace || !al16(workspace) || workspace_bytes < need)) return DREAMER_ERR_ARG;
  return ops::kv4_attn(to_cache(c), ops::Kv4Attn{q, ldq, out, ldo, lens, 0, n_heads, dtype, scale, workspace, status, 0},
                       (cudaStream_t)stream, ops::user_launch((cudaStream_t)stream));
}
