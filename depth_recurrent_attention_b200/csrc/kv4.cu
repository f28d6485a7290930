// A 4-bit cache of attention keys and values: rows quantised as they are written, read back,
// and attended by one query token a sequence.
//
// A group is KV4_GROUP = 64 consecutive channels of one head of one token:
//   s = bf16((max - min) / 15), m = bf16(min), c = min(max(rint((x - m) / s), 0), 15), c = 0
//   where s = 0; the value held is s c + m.  A group with a NaN or a magnitude above 2^126
//   (an infinity) holds s = m = NaN and reads back as NaN.
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
// A CTA takes ROWS_T rows and eight (head, plane) pairs of the keys or of the values
// (blockIdx.z), a warp one of the eight: 8 lanes hold a group's 64 channels, so a warp step is
// four consecutive rows of one (head, plane): 128-byte reads, and 128 contiguous bytes of codes
// and 16 of pairs where the rows are neighbours in a block.
constexpr int ROWS_T = 16;
constexpr int CU_SMEM = 1024;  // boundaries searched in shared memory up to this many sequences

struct RowArgs {
  uint8_t *data;
  int B, Hkv, ng, cap;
  const void *k, *v;
  long ldk, ldv;
  const int *cu, *start;
  int n_rows;
  int zero_rest;  // load: rows of no sequence become zeros
  int *err;
};

// Block offset (in blocks, of head 0) and position in the block of the tile's rows: row r
// belongs to the sequence b with cu[b] <= r < cu[b + 1].  slot < 0: the row is in no sequence,
// or its position is outside the cache (reported).
__device__ __forceinline__ void find_slots(const RowArgs &a, int row0, int *scu, long *blk, int *pos) {
  const int tid = threadIdx.x;
  const int *cu = a.cu;
  if (a.cu && a.B <= CU_SMEM) {
    for (int i = tid; i <= a.B; i += blockDim.x) scu[i] = a.cu[i];
    cu = scu;
  }
  __syncthreads();
  if (tid < ROWS_T) {
    const int r = row0 + tid;
    int p = -1, b = -1, off = 0;
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
          off = r - cu[lo];
        }
      }
      if (b >= 0) {
        const long q = (long)a.start[b] + off;
        if (q >= 0 && q < a.cap) p = (int)q;
        else raise_dev_error(a.err, DEV_BAD_INDEX);
      }
    }
    pos[tid] = p;
    blk[tid] = p < 0 ? 0 : (long)b * a.Hkv * (a.cap / KV4_BLOCK) + p / KV4_BLOCK;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(256) kv4_store_kernel(RowArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int scu[CU_SMEM + 1];
  __shared__ long sblk[ROWS_T];
  __shared__ int spos[ROWS_T];
  const int row0 = blockIdx.x * ROWS_T;
  find_slots(a, row0, scu, sblk, spos);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hp = blockIdx.y * 8 + warp;  // head * ng + plane
  if (hp >= a.Hkv * a.ng) return;
  const int head = hp / a.ng, plane = hp % a.ng;
  const int side = blockIdx.z;
  const T *src = reinterpret_cast<const T *>(side ? a.v : a.k) + (long)hp * KV4_GROUP + (lane & 7) * 8;
  const long ld = side ? a.ldv : a.ldk;
  const int sub = lane >> 3;
  float x[ROWS_T / 4][8];
#pragma unroll
  for (int i = 0; i < ROWS_T / 4; i++)
    if (spos[i * 4 + sub] >= 0) load8(src + (long)(row0 + i * 4 + sub) * ld, x[i]);
  const long head_blk = (long)head * (a.cap / KV4_BLOCK);
  const int block_bytes = a.ng * 2 * (PLANE + PAIRS);
#pragma unroll
  for (int i = 0; i < ROWS_T / 4; i++) {
    const int p = spos[i * 4 + sub];
    if (p < 0) {
#pragma unroll
      for (int e = 0; e < 8; e++) x[i][e] = 0.f;
    }
    float mx = x[i][0], mn = x[i][0], bad = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      mx = fmaxf(mx, x[i][e]);
      mn = fminf(mn, x[i][e]);
      if (!(fabsf(x[i][e]) <= 0x1p126f)) bad = 1.f;  // NaN, infinite or out of range
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, o));
    }
    bf16 sb = __float2bfloat16_rn((float)(((double)mx - (double)mn) / 15.0));
    bf16 mb = __float2bfloat16_rn(mn);
    if (bad != 0.f) sb = mb = __float2bfloat16_rn(NAN);
    const float s = __bfloat162float(sb), m = __bfloat162float(mb);
    uint32_t w = 0;
    if (s > 0.f) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const double qd = ((double)x[i][e] - (double)m) / (double)s;
        const int c = (int)fmin(fmax(rint(qd), 0.0), 15.0);
        w |= (uint32_t)c << (4 * e);
      }
    }
    if (p >= 0) {
      uint8_t *blk = a.data + (sblk[i * 4 + sub] + head_blk) * block_bytes;
      const int t = p % KV4_BLOCK;
      *reinterpret_cast<uint32_t *>(blk + (side * a.ng + plane) * PLANE + t * 32 + (lane & 7) * 4) = w;
      if ((lane & 7) == 0) {
        __nv_bfloat162 pr;
        pr.x = sb;
        pr.y = mb;
        *reinterpret_cast<__nv_bfloat162 *>(blk + 2 * a.ng * PLANE + (side * a.ng + plane) * PAIRS + t * 4) = pr;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) kv4_load_kernel(RowArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int scu[CU_SMEM + 1];
  __shared__ long sblk[ROWS_T];
  __shared__ int spos[ROWS_T];
  const int row0 = blockIdx.x * ROWS_T;
  find_slots(a, row0, scu, sblk, spos);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hp = blockIdx.y * 8 + warp;
  if (hp >= a.Hkv * a.ng) return;
  const int head = hp / a.ng, plane = hp % a.ng;
  const int side = blockIdx.z;
  T *dst = reinterpret_cast<T *>(const_cast<void *>(side ? a.v : a.k)) + (long)hp * KV4_GROUP + (lane & 7) * 8;
  const long ld = side ? a.ldv : a.ldk;
  const int sub = lane >> 3;
  const long head_blk = (long)head * (a.cap / KV4_BLOCK);
  const int block_bytes = a.ng * 2 * (PLANE + PAIRS);
  uint32_t w[ROWS_T / 4];
  float2 sm[ROWS_T / 4];
#pragma unroll
  for (int i = 0; i < ROWS_T / 4; i++) {
    const int p = spos[i * 4 + sub];
    w[i] = 0;
    sm[i] = make_float2(0.f, 0.f);
    if (p < 0) continue;
    const uint8_t *blk = a.data + (sblk[i * 4 + sub] + head_blk) * block_bytes;
    const int t = p % KV4_BLOCK;
    w[i] = *reinterpret_cast<const uint32_t *>(blk + (side * a.ng + plane) * PLANE + t * 32 + (lane & 7) * 4);
    sm[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(
        blk + 2 * a.ng * PLANE + (side * a.ng + plane) * PAIRS + t * 4));
  }
#pragma unroll
  for (int i = 0; i < ROWS_T / 4; i++) {
    if (spos[i * 4 + sub] < 0 && !(a.zero_rest && row0 + i * 4 + sub < a.n_rows)) continue;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e++) x[e] = fmaf(sm[i].x, (float)((w[i] >> (4 * e)) & 15u), sm[i].y);
    store8(dst + (long)(row0 + i * 4 + sub) * ld, x);
  }
}

// ---- attention of one query token a sequence over the cache ------------------------------
// One warp takes whole 64-token blocks, brought in by bulk copies into a ring of its own.
// Products run on warp-level matrix instructions (m16n8k16) with the codes as the A operand:
//   scores   A = 16 keys x 16 channels of K codes, B = channels x 8 columns of q
//   output   A = 16 channels x 16 keys of V codes, B = keys x 8 columns of weights
// A code c enters as the bf16 number c - 8, exact: (0x4300 | c) is 128 + c.  With
// value = s (c - 8) + (m + 8 s), a score is s (q . (c - 8)) + (m + 8 s) sum(q), and a weight p
// enters the output product as p s, the offsets as one sum of p (m + 8 s) a plane.
// A column is (16-key tile of the supertile, query head): GP = 2, 4 or 8 columns hold the query
// heads that share a key head, and 8 / GP key tiles share one accumulator, each with q in its own
// columns and zeros elsewhere.  So one exponential a (key, query head) is computed also where a
// key head has one query head (GP = 2: one idle column of two).  Every column keeps its own
// running maximum and sum; they join at the end: lanes, then warps in shared memory, then the
// CTAs of a cluster (one (sequence, key head) split over the key axis) in distributed shared
// memory.  No workspace, no atomics: the same inputs give the same bits.
//
// The rows r of a 16-key tile are the keys perm(r): with it a warp's 8-byte reads of K rows and
// 4-byte reads of V rows meet every bank once.
struct AttnArgs {
  const uint8_t *data;
  int B, Hkv, cap, Hq, G, qchunks;
  const void *q;
  long ldq;
  void *out;
  long ldo;
  const int *lens;
  int len_add;
  float scale_log2;
  int *err;
};

__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int NG, int GP, int TERMS, int NW, int ST>
struct AttnCfg {
  static constexpr int BLK = NG * 2 * (PLANE + PAIRS);  // bytes of a block
  static constexpr int RING = NW * ST * BLK;
  static constexpr int D = NG * 64;
  // after the loop the ring holds [NW][GP][D] partial outputs
  static constexpr int SMEM = RING > NW * GP * D * 4 ? RING : NW * GP * D * 4;
};

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

template <typename T, int NG, int GP, int TERMS, int NW, int ST>
__global__ void __launch_bounds__(NW * 32) kv4_attn_kernel(AttnArgs a) {
  using C = AttnCfg<NG, GP, TERMS, NW, ST>;
  constexpr int D = C::D;
  constexpr int NTI = 8 / GP;       // key tiles that share an accumulator
  constexpr int NSUP = 4 / NTI;     // accumulators of a block
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[NW * ST];
  __shared__ float sm_m[NW][GP], sm_l[NW][GP];       // of a warp's columns, joined over its tiles
  __shared__ float so[GP][D], sM[GP], sL[GP];        // of the CTA
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
  const int nq = min(GP, a.G - qc * GP);             // query heads of this CTA
  const int head0 = kvh * a.G + qc * GP;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NW * ST; i++) tc::mbar_init(tc::smem_u32(&bars[i]), 1);
    tc::fence_mbar_init();
    s_abort = 0;
  }
  __syncthreads();

  long len = (long)a.lens[b] + a.len_add;
  if (len < 0 || len > a.cap) {                      // reported, and attends to nothing
    if (threadIdx.x == 0) raise_dev_error(a.err, DEV_BAD_INDEX);
    len = 0;
  }
  const int nkeys = (int)len;
  const int nb = (nkeys + KV4_BLOCK - 1) / KV4_BLOCK;
  const int per = (nb + (int)csize - 1) / (int)csize;
  const int blk0 = min(nb, (int)crank * per), blk1 = min(nb, blk0 + per);
  const uint8_t *base = a.data + (long)pair * (a.cap / KV4_BLOCK) * C::BLK;
  const int mine = blk1 - blk0 > warp ? (blk1 - blk0 - warp + NW - 1) / NW : 0;
  uint8_t *wring = ring + warp * ST * C::BLK;
  auto issue = [&](int i) {  // block i of this warp
    const uint32_t bar = tc::smem_u32(&bars[warp * ST + i % ST]);
    tc::mbar_expect_tx(bar, C::BLK);
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(wring + (i % ST) * C::BLK)),
        "l"(base + (long)(blk0 + warp + i * NW) * C::BLK), "r"((uint32_t)C::BLK), "r"(bar)
        : "memory");
  };
  if (lane == 0)
    for (int i = 0; i < ST && i < mine; i++) issue(i);

  // q as B fragments (column g: query head g % GP; channels 16 t .. 16 t + 15 of a plane), in
  // TERMS bf16 terms that add up to q, and sum(q) of a plane for this lane's columns 2t, 2t + 1
  uint32_t qf[NG][8][TERMS];
  float qs[NG][2];
  {
    const int qh = g % GP;
    const T *qp = reinterpret_cast<const T *>(a.q) + (long)b * a.ldq + (long)(head0 + (qh < nq ? qh : 0)) * D + 16 * t;
#pragma unroll
    for (int p = 0; p < NG; p++) {
      float v[16];
      load8(qp + p * 64, v);
      load8(qp + p * 64 + 8, v + 8);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; e++) {
        if (qh >= nq) v[e] = 0.f;
        sum += v[e];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      qs[p][0] = __shfl_sync(0xffffffffu, sum, ((2 * t) % GP) * 4) * a.scale_log2;
      qs[p][1] = __shfl_sync(0xffffffffu, sum, ((2 * t + 1) % GP) * 4) * a.scale_log2;
#pragma unroll
      for (int w = 0; w < 2; w++)
#pragma unroll
        for (int j = 0; j < 4; j++) {  // the order of codes2<j> of word w: elements j and j + 4
          float lo = v[8 * w + j], hi = v[8 * w + j + 4];
#pragma unroll
          for (int k = 0; k < TERMS; k++) {
            const uint32_t pk = bf2_pack_rn(lo, hi);
            qf[p][4 * w + j][k] = pk;
            lo -= __uint_as_float(pk << 16);
            hi -= __uint_as_float(pk & 0xffff0000u);
          }
        }
    }
  }

  float o[NG][4][4];   // [plane][channel tile][c]: channels 8g + mt and 8g + 4 + mt, columns 2t, 2t + 1
  float ofs[NG][2];    // sum of p (m + 8 s)
  float m2[2] = {-INFINITY, -INFINITY}, l2[2] = {0.f, 0.f};
#pragma unroll
  for (int p = 0; p < NG; p++) {
    ofs[p][0] = ofs[p][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 4; mt++)
#pragma unroll
      for (int c = 0; c < 4; c++) o[p][mt][c] = 0.f;
  }
  const int prow = perm_row(g);                       // key of row g of a tile
  const int pv0 = perm_row(2 * t), pv1 = perm_row(2 * t + 1);
  const int my_tile = (2 * t) / GP;                   // tile of this lane's columns
  bool ok = true;
  int done = 0;

  for (int i = 0; i < mine; i++) {
    if (!tc::mbar_wait(tc::smem_u32(&bars[warp * ST + i % ST]), (uint32_t)((i / ST) & 1), (volatile int *)&s_abort, a.err)) {
      ok = false;
      break;
    }
    done = i + 1;
    const uint8_t *blk = wring + (i % ST) * C::BLK;
    const int key0 = (blk0 + warp + i * NW) * KV4_BLOCK;
    const bool tail = key0 + KV4_BLOCK > nkeys;
    // ---- scores
    float x[NSUP][4];
#pragma unroll
    for (int sp = 0; sp < NSUP; sp++) {
#pragma unroll
      for (int c = 0; c < 4; c++) x[sp][c] = 0.f;
#pragma unroll
      for (int p = 0; p < NG; p++) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ti = 0; ti < NTI; ti++) {
          const uint8_t *kr = blk + p * PLANE + ((sp * NTI + ti) * 16 + prow) * 32 + 8 * t;
          const uint2 w0 = *reinterpret_cast<const uint2 *>(kr);
          const uint2 w1 = *reinterpret_cast<const uint2 *>(kr + 8 * 32);
          const bool on = GP == 8 || g / GP == ti;
          const uint32_t ww0[2] = {w0.x, w0.y}, ww1[2] = {w1.x, w1.y};
#pragma unroll
          for (int w = 0; w < 2; w++) {
            uint32_t f0[4] = {codes2<0>(ww0[w]), codes2<0>(ww1[w]), codes2<1>(ww0[w]), codes2<1>(ww1[w])};
            uint32_t f1[4] = {codes2<2>(ww0[w]), codes2<2>(ww1[w]), codes2<3>(ww0[w]), codes2<3>(ww1[w])};
#pragma unroll
            for (int k = TERMS - 1; k >= 0; k--) {
              mma16816(acc, f0, on ? qf[p][4 * w][k] : 0u, on ? qf[p][4 * w + 1][k] : 0u);
              mma16816(acc, f1, on ? qf[p][4 * w + 2][k] : 0u, on ? qf[p][4 * w + 3][k] : 0u);
            }
          }
        }
        const uint8_t *kp = blk + 2 * NG * PLANE + p * PAIRS + ((sp * NTI + my_tile) * 16 + prow) * 4;
        const float2 s0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(kp));
        const float2 s1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(kp + 8 * 4));
        const float u0 = s0.x * a.scale_log2, u1 = s1.x * a.scale_log2;
        const float z0 = fmaf(8.f, s0.x, s0.y), z1 = fmaf(8.f, s1.x, s1.y);
        x[sp][0] += fmaf(u0, acc[0], z0 * qs[p][0]);
        x[sp][1] += fmaf(u0, acc[1], z0 * qs[p][1]);
        x[sp][2] += fmaf(u1, acc[2], z1 * qs[p][0]);
        x[sp][3] += fmaf(u1, acc[3], z1 * qs[p][1]);
      }
      if (tail) {
        const int key = key0 + (sp * NTI + my_tile) * 16 + prow;
        if (key >= nkeys) x[sp][0] = x[sp][1] = -INFINITY;
        if (key + 8 >= nkeys) x[sp][2] = x[sp][3] = -INFINITY;
      }
    }
    // ---- running maximum of the two columns, moved only when it grows by more than 2^8
    float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
    for (int sp = 1; sp < NSUP; sp++) {
      mx0 = fmaxf(mx0, fmaxf(x[sp][0], x[sp][2]));
      mx1 = fmaxf(mx1, fmaxf(x[sp][1], x[sp][3]));
    }
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, k));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, k));
    }
    if (__any_sync(0xffffffffu, mx0 > m2[0] + 8.f || mx1 > m2[1] + 8.f)) {
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
    const float r0 = m2[0] == -INFINITY ? 0.f : m2[0], r1 = m2[1] == -INFINITY ? 0.f : m2[1];
    // ---- weights and output
    float ob[NG][4][4];  // TERMS > 1: the block's own sums, added in 32-bit rounding to nearest
    if (TERMS > 1) {
#pragma unroll
      for (int p = 0; p < NG; p++)
#pragma unroll
        for (int mt = 0; mt < 4; mt++)
#pragma unroll
          for (int c = 0; c < 4; c++) ob[p][mt][c] = 0.f;
    }
#pragma unroll
    for (int sp = 0; sp < NSUP; sp++) {
      const float p0 = tc::ex2(x[sp][0] - r0), p1 = tc::ex2(x[sp][1] - r1);
      const float p2 = tc::ex2(x[sp][2] - r0), p3 = tc::ex2(x[sp][3] - r1);
      l2[0] += p0 + p2;
      l2[1] += p1 + p3;
#pragma unroll
      for (int p = 0; p < NG; p++) {
        const uint8_t *vp = blk + 2 * NG * PLANE + (NG + p) * PAIRS + ((sp * NTI + my_tile) * 16 + prow) * 4;
        float2 s0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(vp));
        float2 s1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(vp + 8 * 4));
        if (tail) {  // what lies behind the last key may be anything
          const int key = key0 + (sp * NTI + my_tile) * 16 + prow;
          if (key >= nkeys) s0 = make_float2(0.f, 0.f);
          if (key + 8 >= nkeys) s1 = make_float2(0.f, 0.f);
        }
        const float z0 = fmaf(8.f, s0.x, s0.y), z1 = fmaf(8.f, s1.x, s1.y);
        ofs[p][0] = fmaf(p0, z0, fmaf(p2, z1, ofs[p][0]));
        ofs[p][1] = fmaf(p1, z0, fmaf(p3, z1, ofs[p][1]));
        uint32_t bq[TERMS][2];  // weights as B fragments: column g, keys perm(2t), perm(2t + 1) (+ 8)
        float y0 = p0 * s0.x, y1 = p1 * s0.x, y2 = p2 * s1.x, y3 = p3 * s1.x;
#pragma unroll
        for (int k = 0; k < TERMS; k++) {
          const uint32_t h0 = bf2_pack_rn(y0, y1), h1 = bf2_pack_rn(y2, y3);
          bq[k][0] = transpose8(h0);
          bq[k][1] = transpose8(h1);
          if (k + 1 < TERMS) {
            y0 -= __uint_as_float(h0 << 16);
            y1 -= __uint_as_float(h0 & 0xffff0000u);
            y2 -= __uint_as_float(h1 << 16);
            y3 -= __uint_as_float(h1 & 0xffff0000u);
          }
        }
#pragma unroll
        for (int ti = 0; ti < NTI; ti++) {
          const uint8_t *vr = blk + (NG + p) * PLANE + (sp * NTI + ti) * 16 * 32 + 4 * g;
          const uint32_t v0 = *reinterpret_cast<const uint32_t *>(vr + pv0 * 32);
          const uint32_t v1 = *reinterpret_cast<const uint32_t *>(vr + pv1 * 32);
          const uint32_t v2 = *reinterpret_cast<const uint32_t *>(vr + (pv0 + 8) * 32);
          const uint32_t v3 = *reinterpret_cast<const uint32_t *>(vr + (pv1 + 8) * 32);
          const uint32_t lo01 = __byte_perm(v0, v1, 0x5410), hi01 = __byte_perm(v0, v1, 0x7632);
          const uint32_t lo23 = __byte_perm(v2, v3, 0x5410), hi23 = __byte_perm(v2, v3, 0x7632);
          const bool on = GP == 8 || g / GP == ti;
          auto tile = [&](auto mtag) {
            constexpr int mt = decltype(mtag)::value;
            const uint32_t f[4] = {codes2<mt>(lo01), codes2<mt>(hi01), codes2<mt>(lo23), codes2<mt>(hi23)};
#pragma unroll
            for (int k = TERMS - 1; k >= 0; k--)
              mma16816(TERMS > 1 ? ob[p][mt] : o[p][mt], f, on ? bq[k][0] : 0u, on ? bq[k][1] : 0u);
          };
          tile(std::integral_constant<int, 0>());
          tile(std::integral_constant<int, 1>());
          tile(std::integral_constant<int, 2>());
          tile(std::integral_constant<int, 3>());
        }
      }
    }
    if (TERMS > 1) {
#pragma unroll
      for (int p = 0; p < NG; p++)
#pragma unroll
        for (int mt = 0; mt < 4; mt++)
#pragma unroll
          for (int c = 0; c < 4; c++) o[p][mt][c] += ob[p][mt][c];
    }
    __syncwarp();
    if (lane == 0 && i + ST < mine) issue(i + ST);  // into the stage just read
  }
  // after an expired wait the copies still in flight land before shared memory is reused
  if (!ok && lane == 0)
    for (int i = done; i < mine && i < done + ST; i++) {
      const uint64_t t0 = tc::globaltimer();
      while (!tc::mbar_try_wait(tc::smem_u32(&bars[warp * ST + i % ST]), (uint32_t)((i / ST) & 1)) &&
             tc::globaltimer() - t0 < tc::WAIT_LIMIT_NS) {
      }
    }

  // ---- join the key tiles' columns of a query head inside the warp
#pragma unroll
  for (int k = 4; k < 32; k <<= 1) {
#pragma unroll
    for (int c = 0; c < 2; c++) {
      l2[c] += __shfl_xor_sync(0xffffffffu, l2[c], k);
#pragma unroll
      for (int p = 0; p < NG; p++) ofs[p][c] += __shfl_xor_sync(0xffffffffu, ofs[p][c], k);
    }
  }
  float M2[2];
#pragma unroll
  for (int c = 0; c < 2; c++) {
    float m = m2[c];
#pragma unroll
    for (int k = GP / 2; k < 4; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    M2[c] = m;
    const float f = m2[c] == -INFINITY ? 0.f : tc::ex2(m2[c] - m);
    // a column with no key yet holds zeros (or what a NaN key left: kept)
    const float ff = m2[c] == -INFINITY ? 1.f : f;
    l2[c] *= ff;
#pragma unroll
    for (int p = 0; p < NG; p++) {
      ofs[p][c] *= ff;
#pragma unroll
      for (int mt = 0; mt < 4; mt++) {
        o[p][mt][c] *= ff;
        o[p][mt][c + 2] *= ff;
      }
    }
#pragma unroll
    for (int k = GP / 2; k < 4; k <<= 1) {
      l2[c] += __shfl_xor_sync(0xffffffffu, l2[c], k);
#pragma unroll
      for (int p = 0; p < NG; p++) {
        ofs[p][c] += __shfl_xor_sync(0xffffffffu, ofs[p][c], k);
#pragma unroll
        for (int mt = 0; mt < 4; mt++) {
          o[p][mt][c] += __shfl_xor_sync(0xffffffffu, o[p][mt][c], k);
          o[p][mt][c + 2] += __shfl_xor_sync(0xffffffffu, o[p][mt][c + 2], k);
        }
      }
    }
  }
  __syncthreads();  // every warp is done with the ring
  float *part = reinterpret_cast<float *>(ring);  // [NW][GP][D]
  if (2 * t < GP) {
#pragma unroll
    for (int c = 0; c < 2; c++) {
      const int qh = 2 * t + c;
      if (g == 0) {
        sm_m[warp][qh] = M2[c];
        sm_l[warp][qh] = l2[c];
      }
#pragma unroll
      for (int p = 0; p < NG; p++)
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          float *dst = part + (warp * GP + qh) * D + p * 64 + 8 * g + 4 * hf;
          *reinterpret_cast<float4 *>(dst) = make_float4(
              o[p][0][c + 2 * hf] + ofs[p][c], o[p][1][c + 2 * hf] + ofs[p][c],
              o[p][2][c + 2 * hf] + ofs[p][c], o[p][3][c + 2 * hf] + ofs[p][c]);
        }
    }
  }
  __syncthreads();
  // ---- join the warps
  for (int e = threadIdx.x; e < GP * D; e += NW * 32) {
    const int qh = e / D;
    float m = sm_m[0][qh];
#pragma unroll
    for (int w = 1; w < NW; w++) m = fmaxf(m, sm_m[w][qh]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float f = sm_m[w][qh] == -INFINITY ? 1.f : tc::ex2(sm_m[w][qh] - m);
      acc = fmaf(f, part[w * GP * D + e], acc);
      l = fmaf(f, sm_l[w][qh], l);
    }
    so[qh][e % D] = acc;
    if (e % D == 0) {
      sM[qh] = m;
      sL[qh] = l;
    }
  }
  // ---- join the CTAs of the cluster: every CTA writes its share of the output
  if (csize > 1) cluster_sync();
  else __syncthreads();
  const int aborted = *(volatile int *)&s_abort;
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
    if (!aborted)
      reinterpret_cast<T *>(a.out)[(long)b * a.ldo + (long)(head0 + qh) * D + e % D] = from_f<T>(res);
  }
  if (csize > 1) cluster_sync();  // shared memory that others read stays until they have
}

template <typename K, typename... A>
int launch(K kern, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s, LaunchOpt o, A... args) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return DREAMER_ERR_CUDA;
  if (cluster > 8 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return DREAMER_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (o.pdl) {
    at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[na].val.programmaticStreamSerializationAllowed = 1;
    na++;
  }
  if (cluster > 1) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = cluster;
    at[na].val.clusterDim.y = 1;
    at[na].val.clusterDim.z = 1;
    na++;
  }
  cfg.attrs = at;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? DREAMER_OK : DREAMER_ERR_CUDA;
}

RowArgs row_args(const Kv4Cache &c, const Kv4Rows &r) {
  RowArgs a{};
  a.data = c.data;
  a.B = c.B; a.Hkv = c.Hkv; a.ng = c.d / KV4_GROUP; a.cap = c.cap;
  a.k = r.k; a.v = r.v; a.ldk = r.ldk; a.ldv = r.ldv;
  a.cu = r.cu; a.start = r.start; a.n_rows = r.n_rows; a.zero_rest = r.zero_rest; a.err = r.err;
  return a;
}
dim3 row_grid(const RowArgs &a) {
  return dim3((a.n_rows + ROWS_T - 1) / ROWS_T, (a.Hkv * a.ng + 7) / 8, 2);
}

template <typename T, int NG, int GP, int TERMS, int NW, int ST>
int launch_attn(const AttnArgs &a, int pairs, int cluster, cudaStream_t s, LaunchOpt o) {
  using C = AttnCfg<NG, GP, TERMS, NW, ST>;
  const long ctas = (long)pairs * a.qchunks * cluster;
  if (ctas > 0x7fffffffL) return DREAMER_ERR_UNSUPPORTED;
  return launch(kv4_attn_kernel<T, NG, GP, TERMS, NW, ST>, dim3((unsigned)ctas), dim3(NW * 32), C::SMEM,
                cluster, s, o, a);
}

template <typename T, int NG, int TERMS>
int dispatch_attn(AttnArgs a, int pairs, int cluster, cudaStream_t s, LaunchOpt o) {
  const int gp = a.G <= 2 ? 2 : a.G <= 4 ? 4 : 8;
  a.qchunks = (a.G + gp - 1) / gp;
  if (gp == 2) return launch_attn<T, NG, 2, TERMS, 4, 3>(a, pairs, cluster, s, o);
  if (gp == 4) return launch_attn<T, NG, 4, TERMS, 4, 3>(a, pairs, cluster, s, o);
  return launch_attn<T, NG, 8, TERMS, 4, 3>(a, pairs, cluster, s, o);
}

}  // namespace

int kv4_store(const Kv4Cache &c, const Kv4Rows &r, cudaStream_t s, LaunchOpt o) {
  if (r.n_rows == 0) return DREAMER_OK;
  const RowArgs a = row_args(c, r);
  return r.dtype == 0 ? launch(kv4_store_kernel<float>, row_grid(a), dim3(256), 0, 1, s, o, a)
                      : launch(kv4_store_kernel<bf16>, row_grid(a), dim3(256), 0, 1, s, o, a);
}

int kv4_load(const Kv4Cache &c, const Kv4Rows &r, cudaStream_t s, LaunchOpt o) {
  if (r.n_rows == 0) return DREAMER_OK;
  const RowArgs a = row_args(c, r);
  return r.dtype == 0 ? launch(kv4_load_kernel<float>, row_grid(a), dim3(256), 0, 1, s, o, a)
                      : launch(kv4_load_kernel<bf16>, row_grid(a), dim3(256), 0, 1, s, o, a);
}

int kv4_attn(const Kv4Cache &c, const Kv4Attn &t, cudaStream_t s, LaunchOpt o) {
  AttnArgs a{};
  a.data = c.data;
  a.B = c.B; a.Hkv = c.Hkv; a.cap = c.cap; a.Hq = t.Hq; a.G = t.Hq / c.Hkv;
  a.q = t.q; a.ldq = t.ldq; a.out = t.out; a.ldo = t.ldo;
  a.lens = t.lens; a.len_add = t.len_add;
  a.scale_log2 = t.scale * 1.4426950408889634f;
  a.err = t.err;
  const int pairs = c.B * c.Hkv;
  // CTAs of a (sequence, key head): enough for several waves, at least four blocks each
  const int nblk = c.cap / KV4_BLOCK;
  int cluster = 1;
  while (cluster < 16 && (long)pairs * cluster < 148 * 8 && nblk / (2 * cluster) >= 4) cluster *= 2;
  const bool f32 = t.dtype == 0;
  if (c.d == 64)
    return f32 ? dispatch_attn<float, 1, 3>(a, pairs, cluster, s, o) : dispatch_attn<bf16, 1, 1>(a, pairs, cluster, s, o);
  return f32 ? dispatch_attn<float, 2, 3>(a, pairs, cluster, s, o) : dispatch_attn<bf16, 2, 1>(a, pairs, cluster, s, o);
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
  return ops::kv4_store(to_cache(c), ops::Kv4Rows{k, v, ldk, ldv, cu_rows, start, n_rows, dtype, 0, status},
                        (cudaStream_t)stream);
}

extern "C" int dreamer_kv4_load(const dreamer_kv4_cache *c, void *k, int64_t ldk, void *v, int64_t ldv,
                                const int32_t *cu_rows, const int32_t *start, int n_rows, int dtype,
                                int zero_rest, int32_t *status, dreamer_stream stream) {
  const int rc = check_rows(c, k, ldk, v, ldv, cu_rows, start, n_rows, dtype);
  if (rc) return rc;
  return ops::kv4_load(to_cache(c), ops::Kv4Rows{k, v, ldk, ldv, cu_rows, start, n_rows, dtype, zero_rest ? 1 : 0, status},
                       (cudaStream_t)stream);
}

extern "C" int dreamer_attn_kv4(const dreamer_kv4_cache *c, const void *q, int64_t ldq, void *out, int64_t ldo,
                                const int32_t *lens, int n_heads, int dtype, float scale, int32_t *status,
                                dreamer_stream stream) {
  const int rc = check_cache(c);
  if (rc) return rc;
  if (!q || !out || !lens || n_heads < 1 || n_heads % c->n_kv_heads || (dtype != 0 && dtype != 1) ||
      !isfinite(scale))
    return DREAMER_ERR_ARG;
  const int es = dtype == 0 ? 4 : 2;
  const int64_t w = (int64_t)n_heads * c->head_dim;
  if (!al16(q) || !al16(out) || ldq < w || ldo < w || (ldq * es) % 16 || (ldo * es) % 16) return DREAMER_ERR_ARG;
  return ops::kv4_attn(to_cache(c), ops::Kv4Attn{q, ldq, out, ldo, lens, 0, n_heads, dtype, scale, status},
                       (cudaStream_t)stream);
}
