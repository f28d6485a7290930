// Causal attention over packed prompts of different lengths, with grouped heads.
//
// Rows of all prompts lie one behind the other; cu[i] .. cu[i + 1] - 1 are prompt i's.  Token t
// of a prompt attends the prompt's tokens up to itself:
//   out[t, h] = sum_{j <= t} softmax_j(scale q[t, h] . k[j, h / G]) v[j, h / G].
//
// Work items are (row tile of a prompt, head).  The host knows the number of rows and prompts
// only, so it launches the most items that they can make, and a block finds its own from cu:
// items are ordered by their tile index, the highest (most keys) first over all prompts, so
// that long items start first and a block's item costs one search over the tile indices with
// the prompts spread over a warp's lanes.
//
// What a row must not see does not touch it, whatever it holds: masked scores are replaced, not
// added to; value rows behind the prompt's end are cleared in shared memory; and where a value
// of the diagonal block is not finite (0 x infinity would reach the rows before it), the block's
// output product is done row by row on CUDA cores up to the row's own position. (The order of its
// float32 sums is another there: the tile's rows may store a neighbouring bfloat16.)
#include <cuda.h>
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

struct PackedArgs {
  const int *cu;
  int n_seq, n_tokens, Hq, G;
  const void *q, *k, *v;  // float32 form
  long ldq, ldk, ldv;
  void *out;
  long ldo;
  const int *out_rows;    // output row of token t, or null: t
  float scale_log2;
  int *err;
#ifdef DREAMER_TEST_HOOKS
  Withhold withhold;      // of the K (warp 0) or V (warp 2) blocks
#endif
};

// First row and length of prompt i; boundaries outside 0 .. n_tokens are cut, and an end before its start.
// Boundaries that decrease (reported) can leave rows in two prompts, whose blocks then both write them.
__device__ __forceinline__ int2 prompt_rows(const PackedArgs &a, int i) {
  const int lo = min(max(a.cu[i], 0), a.n_tokens);
  const int hi = min(max(a.cu[i + 1], lo), a.n_tokens);
  return make_int2(lo, hi - lo);
}

// Item `rank` (a warp calls it): {first row, length, tile}, or tile < 0 when there are fewer items.
// ge(p) = number of (prompt, tile) with a tile index >= p decreases in p: the item's tile index
// is the p with ge(p + 1) <= rank < ge(p), and its prompt the (rank - ge(p + 1))-th that has
// more than p tiles.
//
// With more than MANY prompts that search would outlast their attention.  There item r is tile
// r - s(i) of the last prompt i with s(i) = cu[i] / ROWS + i <= r, in the prompts' order: s grows by at
// least the number of a prompt's tiles, and a search by 32 takes three or four steps.  8 heads of 64,
// bfloat16: 65 prompts of up to 512 tokens 46 us against 50, 2048 of up to 15 tokens 316 against 752; with
// fewer prompts starting the long ones first is worth more (64 of up to 2048, 2 heads: 71 against 63).
constexpr int MANY = 64;
template <int ROWS>
__device__ __forceinline__ int3 find_item(const PackedArgs &a, int rank) {
  const int lane = threadIdx.x & 31;
  if (a.n_seq > MANY) {
    int lo = 0, hi = a.n_seq;  // lo: s(lo) <= rank, or none
    for (;;) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const unsigned upto = __ballot_sync(0xffffffffu, i < hi && prompt_rows(a, i).x / ROWS + i <= rank);
      if (!(upto & 1u)) return make_int3(0, 0, -1);
      lo += (31 - __clz(upto)) * step;
      hi = min(hi, lo + step);
      if (step == 1) break;
    }
    const int2 pr = prompt_rows(a, lo);
    const int t = rank - pr.x / ROWS - lo;
    return make_int3(pr.x, pr.y, t < (pr.y + ROWS - 1) / ROWS ? t : -1);
  }
  int first = 0;  // tiles of this lane's first prompt (lane): the others are read again
  int most = 0;
  for (int i = lane; i < a.n_seq; i += 32) {
    const int n = (prompt_rows(a, i).y + ROWS - 1) / ROWS;
    if (i == lane) first = n;
    most = max(most, n);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  auto ge = [&](int p) {
    int s = max(0, first - p);
    for (int i = lane + 32; i < a.n_seq; i += 32)
      s += max(0, (prompt_rows(a, i).y + ROWS - 1) / ROWS - p);
    return __reduce_add_sync(0xffffffffu, s);
  };
  if (rank >= ge(0)) return make_int3(0, 0, -1);
  int lo = 0, hi = most - 1;  // the highest p with ge(p) > rank
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ge(mid) > rank) lo = mid;
    else hi = mid - 1;
  }
  int left = rank - ge(lo + 1);
  for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
    const int i = i0 + lane;
    const int2 pr = i < a.n_seq ? prompt_rows(a, i) : make_int2(0, 0);
    const unsigned has = __ballot_sync(0xffffffffu, (pr.y + ROWS - 1) / ROWS > lo);
    const int n = __popc(has);
    if (left < n) {
      const unsigned below = (1u << lane) - 1;
      const int src = __ffs(__ballot_sync(0xffffffffu, ((has >> lane) & 1) && __popc(has & below) == left)) - 1;
      return make_int3(__shfl_sync(0xffffffffu, pr.x, src), __shfl_sync(0xffffffffu, pr.y, src), lo);
    }
    left -= n;
  }
  return make_int3(0, 0, -1);
}

// boundaries that are not 0 <= cu[0] <= ... <= cu[n_seq] <= n_tokens are reported
__device__ __forceinline__ void check_cu(const PackedArgs &a) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int i = lane; i < a.n_seq; i += 32) bad |= a.cu[i] < 0 || a.cu[i + 1] < a.cu[i] || a.cu[i + 1] > a.n_tokens;
  if (bad) raise_dev_error(a.err, DEV_BAD_INDEX);
}

// ---- bfloat16: tcgen05 ---------------------------------------------------------------------
// An SM holds two 128-query tiles: at head dim 128 one CTA takes two adjacent tiles A, B of a prompt and
// a head that share every K/V block; at 64 there are two CTAs of one tile (A) each, and while one starts
// or ends its item the other computes (8 ragged prompts of up to 2048 tokens, 16 heads: 66.4 -> 63.2 us;
// one prompt of 8192: 244 -> 242 under the power cap, 215 at 1965 MHz).  Warp 0 loads Q and K by TMA, warp
// 2 V, warp 1 issues the MMAs, warps 4 and up hold one query row a thread.
// Scores, weights and outputs stay in tensor memory; the output is rescaled only when a row's maximum
// grows by more than 2^8.  Weights enter the output product as bf16 (half a step of 2^-8 relative each, as
// the stored output is), their sum is of the float32 values.
//
// What bounds it, in cycles of a block of 128 x 128 and one tile, by clocks read in the kernel: at head
// dim 128 the products take 1020 and the row's part (scores out, maximum, exponentials, weights in) 1750,
// one after the other for a tile, which two tiles overlap in part; at head dim 64 the products take
// 960 and the row's parts of both tiles together 2900, of which the exponentials' unit is busy 2048.
// An item costs 8000 to 10000 cycles beside its blocks (its place in the batch found, first loads and
// scores, last product and output), which is what short prompts are bound by.
// So
//   - head dim 64 keeps the weights in tensor-memory columns of their own, and the next block's
//     scores are computed as soon as this block's are in registers (one sequence of 8192 tokens, 16
//     heads of 64, two tiles a CTA: 248 -> 231 us at one clock); at 128 tensor memory is full, the weights
//     lie over their scores;
//   - the products are issued by a converged warp's elected lane (3 to 6 % against one lane of a split
//     warp).
// A polynomial for a part of the exponentials (2 to 5 of every 8 pairs) cost 1 to 14 %, the weights handed
// over in halves 4 %: neither is taken.
template <int D>
struct PkCfg {
  static constexpr int CH = D / 64;                 // 64-column chunks of a head
  static constexpr int TILE = 128 * 128;            // bytes of one [128 x 64] bf16 chunk
  static constexpr int TILES = D == 64 ? 1 : 2;     // query tiles of a CTA
  static constexpr int CTAS = D == 64 ? 2 : 1;      // CTAs of an SM
  static constexpr int THREADS = 128 + 128 * TILES;
  static constexpr int COLS = 512 / CTAS;           // tensor-memory columns
  static constexpr int KST = D == 64 ? 3 : 2;       // K ring depth
  static constexpr int VST = 2;                     // V ring depth
  static constexpr int Q_BYTES = TILES * CH * TILE;
  static constexpr int KV_BYTES = CH * TILE;        // one K (or V) block
  static constexpr int SMEM = Q_BYTES + (KST + VST) * KV_BYTES + 1024 + 256;
  static constexpr bool SEP = D == 64;              // weights in columns of their own
  // columns of tile t: scores t * 128, weights P0 + t * 128, output O0 + t * D
  static constexpr int P0 = SEP ? 128 : 0, O0 = SEP ? 192 : 256;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "smem");
};
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r) : "r"(taddr) : "memory");
  return r;
}

// one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// D[tmem] (+)= A B^T with the descriptors' low words (address and leading offset) and common high word:
// A in shared memory, or in tensor memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(PkCfg<D>::THREADS, PkCfg<D>::CTAS)
    packed_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, PackedArgs a) {
  using namespace tc;
  using C = PkCfg<D>;
  constexpr int CH = C::CH, KST = C::KST, VST = C::VST;
  constexpr bool SEP = C::SEP;
  constexpr int TILES = C::TILES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = smem;
  uint8_t *sK = sQ + C::Q_BYTES;
  uint8_t *sV = sK + KST * C::KV_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sV + VST * C::KV_BYTES);
  uint64_t *q_full = bars;
  uint64_t *k_full = q_full + 1, *k_empty = k_full + KST;
  uint64_t *v_full = k_empty + KST, *v_empty = v_full + VST;
  // per tile: scores ready; SEP: scores in registers; weights ready; SEP: output product done
  uint64_t *s_full = v_empty + VST, *s_read = s_full + 2, *p_full = s_read + 2, *pv_done = p_full + 2;
  uint64_t *drained = pv_done + 2;  // after an expired wait: no product is in flight
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *item_slot = reinterpret_cast<int *>(tmem_slot + 2);          // row0, length, tile
  volatile int *by_rows = reinterpret_cast<volatile int *>(tmem_slot + 5);  // [2] diagonal block on CUDA cores

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % a.Hq;
  if (threadIdx.x == 64) {
    mbar_init(smem_u32(q_full), 1);
    for (int s = 0; s < KST; s++) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
    }
    for (int s = 0; s < VST; s++) {
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_read[i]), 4);
      mbar_init(smem_u32(&p_full[i]), 4);
      mbar_init(smem_u32(&pv_done[i]), 1);
      by_rows[i] = 0;
    }
    mbar_init(smem_u32(drained), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmq);
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  pdl_wait();  // inputs of the previous kernel are visible from here on
  // tensor memory only now: a kernel before, of whatever origin, may have to allocate its own yet
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::COLS);
    tmem_relinquish();
  }
  if (warp == 0) {
    if (blockIdx.x == 0) check_cu(a);
    const int3 it = find_item<128 * TILES>(a, blockIdx.x / a.Hq);
    if (lane == 0) {
      item_slot[0] = it.x;
      item_slot[1] = it.y;
      item_slot[2] = it.z;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // after the TMEM allocation (see pdl_trigger)
  const uint32_t tmem = *tmem_slot;
  const int row0 = item_slot[0], S = item_slot[1], pair = item_slot[2];
  if (pair < 0) {  // fewer items than launched
    if (warp == 1) tmem_dealloc(tmem, C::COLS);
    return;
  }
  const int qtA = TILES * pair, qtB = qtA + 1;
  const bool hasB = TILES == 2 && qtB * 128 < S;
  const int nbA = qtA + 1, nbB = hasB ? qtB + 1 : 0;
  const int nb = hasB ? nbB : nbA;
  const uint32_t tS = tmem, tP = tmem + C::P0, tO = tmem + C::O0;

  // Registers as the warps need them, of the launch's 256 x 128: 128 x 56 and 128 x 200
  if (warp < 4) {
    if (TILES == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------- producers (warp 0: Q, K; warp 2: V)
      if (lane == 0) {
        const bool isK = warp == 0;
        const int colb = (head / a.G) * D;
        if (isK) {
          mbar_expect_tx(smem_u32(q_full), (hasB ? 2 : 1) * CH * C::TILE);
          for (int t = 0; t < (hasB ? 2 : 1); t++)
            for (int c = 0; c < CH; c++)
              tma_load_2d(smem_u32(sQ + (t * CH + c) * C::TILE), &tmq, smem_u32(q_full), head * D + 64 * c,
                          row0 + (t == 0 ? qtA : qtB) * 128);
        }
        const CUtensorMap *tm = isK ? &tmk : &tmv;
        const int NS = isK ? KST : VST;
        uint64_t *fullb = isK ? k_full : v_full, *emptyb = isK ? k_empty : v_empty;
        uint8_t *ring = isK ? sK : sV;
        int issued_ph[4] = {-1, -1, -1, -1};
        for (int j = 0; j < nb; j++) {
          const int s = j % NS;
          const uint32_t ph = (j / NS) & 1;
          if (!mbar_wait(smem_u32(&emptyb[s]), ph ^ 1, abort_flag, a.err)) break;
          mbar_expect_tx(smem_u32(&fullb[s]), C::KV_BYTES);
#ifdef DREAMER_TEST_HOOKS
          if (j == a.withhold.copy_of(blockIdx.x, warp)) continue;
#endif
          for (int c = 0; c < CH; c++)
            tma_load_2d(smem_u32(ring + s * C::KV_BYTES + c * C::TILE), tm, smem_u32(&fullb[s]),
                        colb + 64 * c, row0 + j * 128);
          issued_ph[s] = (int)ph;
        }
        // every copy issued lands before the CTA can exit, also where another warp gave up waiting
        const uint64_t t0 = globaltimer();
        if (isK)
          while (!mbar_try_wait(smem_u32(q_full), 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
          }
        for (int i = 0; i < NS; i++)
          if (issued_ph[i] >= 0) {
            const uint64_t t1 = globaltimer();
            while (!mbar_try_wait(smem_u32(&fullb[i]), (uint32_t)issued_ph[i]) &&
                   globaltimer() - t1 < WAIT_LIMIT_NS) {
            }
          }
      }
    } else if (warp == 1) {
      // ------------------------------------------------- MMA issuer
      // Per tile S(0); then for each block j (SEP) S(j+1) once S(j) is in registers and P(j) V_j once the
      // weights are ready, or P(j) V_j and then S(j+1) over them.  The whole warp walks the loop with
      // values that are the same in every lane and one elected lane issues: a chain of descriptors
      // computed by one thread of a split warp took longer than the products.
      constexpr uint32_t ID_S = idesc_bf16_m128(128);
      constexpr uint32_t ID_PV = idesc_bf16_m128_bmn(D);
      constexpr uint32_t DESC_HI = (1024 >> 4) | 1u << 14 | 2u << 29;  // 8-row groups 1024 bytes apart, SW128
      const int uA = __shfl_sync(0xffffffffu, nbA, 0), uB = __shfl_sync(0xffffffffu, nbB, 0);
      const int un = max(uA, uB);
      const uint32_t ut = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = smem_u32(sQ) >> 4 | 1u << 16, k_lo = smem_u32(sK) >> 4 | 1u << 16;
      const uint32_t v_lo = smem_u32(sV) >> 4 | (uint32_t)(C::TILE >> 4) << 16;
      const bool one = elect_one();
      auto wait = [&](uint64_t *bar, int n) {
        const bool r = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), n & 1, abort_flag, a.err));
        tc_fence_after();
        return r;
      };
      auto commit = [&](uint64_t *bar) {
        if (one) mma_commit(smem_u32(bar));
      };
      auto issue_s = [&](int t, int ks) {
        if (one) {
#pragma unroll
          for (int k = 0; k < D / 16; k++) {
            const uint32_t off = ((k >> 2) * C::TILE + (k & 3) * 32) >> 4;
            mma_ss(ut + t * 128, q_lo + ((t * CH * C::TILE) >> 4) + off, k_lo + ks * (C::KV_BYTES >> 4) + off, DESC_HI, ID_S, k != 0);
          }
        }
      };
      auto issue_pv = [&](int t, int j, int vs) {  // 128 keys, 16 per instruction (8 TMEM columns of P)
        if (j + 1 == (t == 0 ? uA : uB) && by_rows[t]) return;
        if (one) {
#pragma unroll
          for (int k = 0; k < 8; k++)
            mma_ts(ut + C::O0 + t * D, ut + C::P0 + t * 128 + k * 8, v_lo + vs * (C::KV_BYTES >> 4) + k * 128, DESC_HI,
                   ID_PV, k == 0 ? (uint32_t)j : 1u);
        }
      };
      bool ok = wait(q_full, 0) && wait(&k_full[0], 0);
      if (ok) {
        issue_s(0, 0);
        commit(&s_full[0]);
        if (uB > 0) {
          issue_s(1, 0);
          commit(&s_full[1]);
        }
        commit(&k_empty[0]);
      }
      int vs = 0, ks = 1 % KST;  // stages of block j's values and of block j + 1's keys
      int j = 0;
      for (; j < un && ok; j++) {
        const bool next = j + 1 < un;
        if (SEP && next) {
          if (!wait(&k_full[ks], (j + 1) / KST)) break;
#pragma unroll
          for (int t = 0; t < TILES; t++)
            if (ok && j + 1 < (t == 0 ? uA : uB)) {
              ok = wait(&s_read[t], j);
              if (ok) issue_s(t, ks);
              if (ok) commit(&s_full[t]);
            }
          if (ok) commit(&k_empty[ks]);
        }
        if (!ok || !wait(&v_full[vs], j / VST)) break;
        if (!SEP && next && !wait(&k_full[ks], (j + 1) / KST)) break;
#pragma unroll
        for (int t = 0; t < TILES; t++)
          if (ok && j < (t == 0 ? uA : uB)) {
            ok = wait(&p_full[t], j);
            if (!ok) break;
            issue_pv(t, j, vs);
            if (!SEP && j + 1 < (t == 0 ? uA : uB)) issue_s(t, ks);
            commit(SEP ? &pv_done[t] : &s_full[t]);
          }
        if (!ok) break;
        commit(&v_empty[vs]);
        if (!SEP && next) commit(&k_empty[ks]);
        if (++vs == VST) vs = 0;
        if (++ks == KST) ks = 0;
      }
      if (j < un || !ok) {  // gave up: the products issued end before tensor memory is given back
        commit(drained);
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(drained), 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
        }
      }
    }
  } else {
    if (TILES == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ------------------------------------------------- softmax (tile A: warps 4-7, B: 8-11)
    const int t = warp < 8 ? 0 : 1;
    const int nbt = t == 0 ? nbA : nbB;
    const int qt = t == 0 ? qtA : qtB;
    if (nbt > 0) {
      const int q = warp & 3;
      const int row = q * 32 + lane;
      const int qi = qt * 128 + row;               // query position in the prompt
      const uint32_t lane_off = (uint32_t)(q * 32) << 16;
      const uint32_t sbuf = tS + t * 128 + lane_off;
      const uint32_t pbuf = tP + t * 128 + lane_off;
      const uint32_t obuf = tO + t * D + lane_off;
      // the same answer in every lane: what follows is done by whole warps
      auto wait_warp = [&](uint64_t *bar, int n) {
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), n & 1, abort_flag, a.err));
      };
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nbt; j++) {
        const bool diag = (j == qt);
        if (diag) {
          // the diagonal block's values: rows behind the prompt's end are cleared, and a value
          // that is not finite sends the block's output product to the row form below
          ok = wait_warp(&v_full[j % VST], j / VST);
          bool bad = false;
          if (ok) {
            uint8_t *vr = sV + (j % VST) * C::KV_BYTES + row * 128;
            if (qi >= S) {
#pragma unroll
              for (int c = 0; c < CH * 8; c++)
                *reinterpret_cast<uint4 *>(vr + (c >> 3) * C::TILE + ((c + row) & 7) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async();
            } else {
              __nv_bfloat162 z = __float2bfloat162_rn(0.f), acc = z;  // x * 0 is NaN where x is not finite
#pragma unroll
              for (int c = 0; c < CH * 8; c++) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vr + (c >> 3) * C::TILE + ((c + row) & 7) * 16);
                const __nv_bfloat162 *h2 = reinterpret_cast<const __nv_bfloat162 *>(&w);
#pragma unroll
                for (int e = 0; e < 4; e++) acc = __hfma2(h2[e], z, acc);
              }
              const uint32_t u = *reinterpret_cast<const uint32_t *>(&acc);
              bad = (u & 0x7fff7fffu) != 0;
            }
          }
          if (bad) by_rows[t] = 1;  // seen by the MMA warp through p_full, by this warp at the end
          if (!ok) break;
        }
        if (!wait_warp(&s_full[t], j)) { ok = false; break; }
        tc_fence_after();
        const int lim = qi - j * 128;  // diagonal block: last visible key of the row
        // the row's 128 scores into registers with four loads in flight
        float sv[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32_async(sbuf + c, sv + c);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld_fence(sv + c);
        if (SEP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_read[t]));
        }
        if (diag) {
#pragma unroll
          for (int i = 0; i < 128; i++)
            if (i > lim) sv[i] = -INFINITY;
        }
        // row max of the raw scores (the scale is positive: applied to the max)
        float mc[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int k = 0; k < 4; k++) mc[k] = max3f(mc[k], sv[i + 2 * k], sv[i + 2 * k + 1]);
        mc[0] = max3f(mc[0], sv[124], sv[125]);
        mc[1] = max3f(mc[1], sv[126], sv[127]);
        const float mraw = max3f(mc[0], mc[1], fmaxf(mc[2], mc[3]));
        const float mx = mraw * a.scale_log2;
        // lazy rescale: move the reference max only when the row max grows by more than 8
        float m_new = m_ref, alpha = 1.f;
        if (mx > m_ref + 8.f) {
          m_new = mx;
          alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - mx);
        }
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        // P = 2^(s * scale - m) as bf16 pairs (the lower key in the low half), where the P.V MMA
        // reads it, and summed
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nm2 = f2_pack(-m_use, -m_use);
        uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};  // four independent sums of pairs
#pragma unroll
        for (int hh = 0; hh < 2; hh++) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; e++) {
            const int i = hh * 64 + 2 * e;
            const float2 x = f2_unpack(f2_fma(f2_pack(sv[i], sv[i + 1]), sc2, nm2));
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            rs2[e & 3] = f2_add(rs2[e & 3], f2_pack(p0, p1));
            w[e] = bf2_pack_rn(p0, p1);
          }
          if (hh == 0) {
            // P V of block j - 1 is done with the weights, and O holds it (else: s_full said so)
            if (SEP && j > 0) {
              ok = wait_warp(&pv_done[t], j - 1);
              tc_fence_after();
            }
            // O rescaled before P(j) V accumulates into it
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float ov[32];
                tmem_ld32(obuf + c, ov);
#pragma unroll
                for (int i = 0; i < 32; i++) ov[i] *= alpha;
                tmem_st32(obuf + c, ov);
              }
            }
          }
          tmem_st32_nowait(pbuf + hh * 32, w);
        }
        const float2 rsf = f2_unpack(f2_add(f2_add(rs2[0], rs2[1]), f2_add(rs2[2], rs2[3])));
        l = l * alpha + rsf.x + rsf.y;
        m_ref = m_new;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[t]));
        if (!ok) break;
      }
      // the commit after the last P.V: O_t is final
      if (ok && wait_warp(SEP ? &pv_done[t] : &s_full[t], SEP ? nbt - 1 : nbt)) {
        tc_fence_after();
        const float inv = 1.0f / l;
        const bool slow = by_rows[t] != 0;
        const uint8_t *vlast = sV + ((nbt - 1) % VST) * C::KV_BYTES;
        const int trow = row0 + qi;
        const bool mine = qi < S;
        const long orow = mine && a.out_rows ? a.out_rows[trow] : trow;
        bf16 *dst = reinterpret_cast<bf16 *>(a.out) + orow * a.ldo + head * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float ov[32];
          __syncwarp();
          if (!slow || nbt > 1) {
            tmem_ld32(obuf + c, ov);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i++) ov[i] = 0.f;
          }
          if (slow) {  // the diagonal block, keys 0 .. row, two a step
            const uint8_t *vc = vlast + (c >> 6) * C::TILE;
#pragma unroll 1
            for (int kp = 0; kp < 64; kp++) {
              __syncwarp();
              const uint32_t pw = tmem_ld1(pbuf + kp);
#pragma unroll
              for (int hf = 0; hf < 2; hf++) {
                const int key = 2 * kp + hf;
                if (key > row) continue;
                const float p = __uint_as_float(hf ? pw & 0xffff0000u : pw << 16);
#pragma unroll
                for (int x = 0; x < 4; x++) {
                  float v8[8];
                  load8(reinterpret_cast<const bf16 *>(vc + key * 128 + ((((c & 63) >> 3) + x) ^ (key & 7)) * 16), v8);
#pragma unroll
                  for (int e = 0; e < 8; e++) ov[8 * x + e] = fmaf(p, v8[e], ov[8 * x + e]);
                }
              }
            }
          }
          if (mine) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float t8[8];
#pragma unroll
              for (int e = 0; e < 8; e++) t8[e] = ov[i + e] * inv;
              store8(dst + c + i, t8);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// ---- float32: CUDA cores -------------------------------------------------------------------
// A CTA takes one head and 32 query rows of a prompt; its groups of 128 threads take the 64-key
// blocks in turns, each with its own softmax and buffers (one group's loads run beside the
// others' arithmetic, and a long row's chain of blocks is cut by their number), and join at the end.  A
// group's threads form an 8 x 16 grid: 4 rows x 4 keys (tx, tx + 16, ..) of the scores and 4 rows x
// D / 16 columns of the output each.  Q and K rows are padded by 4 words, so that eight rows' 16-byte
// reads meet every bank once; a step of 4 channels reads eight words of 16 bytes for 64 multiply-adds,
// issued as 32 of pairs (359 -> 345 us, 8 prompts of up to 2000 tokens, 8 heads of 64: half of the
// multiply-add rate, bound by issue and shared memory; copies a block ahead measured no faster).
//
// Two groups a CTA and two CTAs an SM (one at head dim 128); four groups and one CTA where the items
// would not keep that many busy, and the chain of the longest row decides (long_chains).
template <int D, int NG>
struct F32Cfg {
  static constexpr int BM = 32, BN = 64;
  static constexpr int GROUPS = NG;  // of 128 threads
  static constexpr int CTAS = D <= 64 && NG == 2 ? 2 : 1;
  static constexpr int THREADS = 128 * GROUPS;
  static constexpr int RP = D + 4;   // padded row of Q and K
  static constexpr int PP = BM + 4;  // padded row of the weights [key][row]
  static constexpr int GROUP = BN * RP + BN * D + BN * PP;  // floats of a group's K, V, weights
  static constexpr int SMEM = (BM * RP + GROUPS * GROUP) * 4;
};

template <int D, int NG>
__global__ void __launch_bounds__(F32Cfg<D, NG>::THREADS, F32Cfg<D, NG>::CTAS) packed_f32_kernel(PackedArgs a) {
  using C = F32Cfg<D, NG>;
  constexpr int BM = C::BM, BN = C::BN, RP = C::RP, PP = C::PP;
  constexpr int OC = D / 16;  // output columns of a thread
  constexpr int KJ = BN / 16;  // and keys of a block
  constexpr int GROUPS = C::GROUPS;
  extern __shared__ __align__(16) float fsm[];
  __shared__ int item[3];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x >> 7, tid = threadIdx.x & 127;
  float *sQ = fsm;                                // [BM][RP]
  float *sK = fsm + BM * RP + group * C::GROUP;   // [BN][RP]
  float *sV = sK + BN * RP;                       // [BN][D]
  float *sP = sV + BN * D;                        // [BN][PP]
  const int head = blockIdx.x % a.Hq, kvh = head / a.G;
  if (threadIdx.x < 32) {
    if (blockIdx.x == 0) check_cu(a);
    const int3 it = find_item<BM>(a, blockIdx.x / a.Hq);
    if (threadIdx.x == 0) {
      item[0] = it.x;
      item[1] = it.y;
      item[2] = it.z;
    }
  }
  __syncthreads();
  const int row0 = item[0], S = item[1], tile = item[2];
  if (tile < 0) return;
  const int q0 = tile * BM;
  const int ty = tid >> 4, tx = tid & 15;
  // rows n of a [rows][D] matrix into padded rows; rows that do not exist become zeros
  auto fetch = [&](const void *src, long ld, int first, int rows, int col, float *dst, int pitch, int t, int step) {
    const float *g = reinterpret_cast<const float *>(src) + (long)row0 * ld + col;
    for (int e = t; e < rows * (D / 4); e += step) {
      const int r = e / (D / 4), c = e % (D / 4);
      const bool in = first + r < S;
      tc::cp_async16(tc::smem_u32(dst + r * pitch + 4 * c), g + (long)(in ? first + r : 0) * ld + 4 * c, in ? 16u : 0u);
    }
  };
  auto landed = [] { asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory"); };
  auto group_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };
  fetch(a.q, a.ldq, q0, BM, head * D, sQ, RP, threadIdx.x, C::THREADS);
  landed();
  __syncthreads();
  float o[4][OC], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < OC; c++) o[i][c] = 0.f;
  }
  const int last = min(S, q0 + BM);  // keys of the tile's last row
  for (int k0 = group * BN; k0 < last; k0 += GROUPS * BN) {
    group_sync();  // the block before is done with
    fetch(a.k, a.ldk, k0, BN, kvh * D, sK, RP, tid, 128);
    fetch(a.v, a.ldv, k0, BN, kvh * D, sV, D, tid, 128);
    landed();
    group_sync();
    float s[4][KJ];
    {
      uint64_t s2[4][KJ];  // sums of even and of odd channels
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < KJ; j++) s2[i][j] = 0ull;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        ulonglong2 qa[4], ka[KJ];
#pragma unroll
        for (int i = 0; i < 4; i++) qa[i] = *reinterpret_cast<const ulonglong2 *>(sQ + (4 * ty + i) * RP + d);
#pragma unroll
        for (int j = 0; j < KJ; j++) ka[j] = *reinterpret_cast<const ulonglong2 *>(sK + (tx + 16 * j) * RP + d);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < KJ; j++) s2[i][j] = f2_fma(qa[i].y, ka[j].y, f2_fma(qa[i].x, ka[j].x, s2[i][j]));
      }
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < KJ; j++) {
          const float2 u = f2_unpack(s2[i][j]);
          s[i][j] = u.x + u.y;
        }
    }
    const bool diag = k0 + BN > q0;  // some key of the block is behind some row
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < KJ; j++) {
        s[i][j] *= a.scale_log2;
        if (diag && k0 + tx + 16 * j > q0 + 4 * ty + i) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float alpha = m[i] == -INFINITY ? 0.f : exp2f(m[i] - base);
      float ps = 0.f;
#pragma unroll
      for (int j = 0; j < KJ; j++) {
        s[i][j] = exp2f(s[i][j] - base);
        ps += s[i][j];
      }
      if (mn != m[i]) {
        l[i] *= alpha;
#pragma unroll
        for (int c = 0; c < OC; c++) o[i][c] *= alpha;
      }
      l[i] += ps;
      m[i] = mn;
    }
#pragma unroll
    for (int j = 0; j < KJ; j++)
      *reinterpret_cast<float4 *>(sP + (tx + 16 * j) * PP + 4 * ty) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncwarp();  // a row's weights are written and read by the same half warp
    const int nk = min(BN, last - k0);
    auto out_step = [&](int k, auto dtag) {
      constexpr bool DIAG = decltype(dtag)::value;
      const float4 pv = *reinterpret_cast<const float4 *>(sP + k * PP + 4 * ty);
      const float pa[4] = {pv.x, pv.y, pv.z, pv.w};
      float va[OC];
      if constexpr (OC >= 4) {
#pragma unroll
        for (int c = 0; c < OC / 4; c++) {
          const float4 w = *reinterpret_cast<const float4 *>(sV + k * D + c * 64 + 4 * tx);
          va[4 * c] = w.x; va[4 * c + 1] = w.y; va[4 * c + 2] = w.z; va[4 * c + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < OC; c++) va[c] = sV[k * D + OC * tx + c];
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (DIAG && k0 + k > q0 + 4 * ty + i) continue;  // 0 x infinity stays out
        if constexpr (OC >= 2) {
#pragma unroll
          for (int c = 0; c < OC; c += 2) {
            const float2 u = f2_unpack(f2_fma(f2_pack(pa[i], pa[i]), f2_pack(va[c], va[c + 1]), f2_pack(o[i][c], o[i][c + 1])));
            o[i][c] = u.x;
            o[i][c + 1] = u.y;
          }
        } else {
          o[i][0] = fmaf(pa[i], va[0], o[i][0]);
        }
      }
    };
    if (!diag) {
#pragma unroll 8
      for (int k = 0; k < BN; k++) out_step(k, std::false_type());
    } else {
#pragma unroll 2
      for (int k = 0; k < nk; k++) out_step(k, std::true_type());
    }
  }
  // the other groups' sums over their own buffers, where the first one takes them in
  static_assert(C::GROUP >= (4 * OC + 8) * 128, "join buffer");
  if (group > 0) {
    float *x = sK;  // [4 * OC + 8][128]
    group_sync();
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
      for (int c = 0; c < OC; c++) x[(i * OC + c) * 128 + tid] = o[i][c];
      x[(4 * OC + i) * 128 + tid] = m[i];
      x[(4 * OC + 4 + i) * 128 + tid] = l[i];
    }
  }
  __syncthreads();
  if (group > 0) return;
  const int groups = min(GROUPS, (last + BN - 1) / BN);  // those with a key
#pragma unroll
  for (int i = 0; i < 4; i++) {
    for (int gr = 1; gr < groups; gr++) {
      const float *x = sK + gr * C::GROUP;
      const float m1 = x[(4 * OC + i) * 128 + tid], mn = fmaxf(m[i], m1);
      // a group without a visible key holds zeros
      const float f0 = m[i] == -INFINITY ? 1.f : exp2f(m[i] - mn), f1 = m1 == -INFINITY ? 1.f : exp2f(m1 - mn);
      l[i] = fmaf(f1, x[(4 * OC + 4 + i) * 128 + tid], l[i] * f0);
#pragma unroll
      for (int c = 0; c < OC; c++) o[i][c] = fmaf(f1, x[(i * OC + c) * 128 + tid], o[i][c] * f0);
      m[i] = mn;
    }
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
    const int r = q0 + 4 * ty + i;
    if (r >= S) continue;
    const long orow = a.out_rows ? a.out_rows[row0 + r] : row0 + r;
    float *dst = reinterpret_cast<float *>(a.out) + orow * a.ldo + (long)head * D;
    const float inv = 1.0f / l[i];
    if constexpr (OC >= 4) {
#pragma unroll
      for (int c = 0; c < OC / 4; c++)
        *reinterpret_cast<float4 *>(dst + c * 64 + 4 * tx) = make_float4(
            o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
    } else {
#pragma unroll
      for (int c = 0; c < OC; c++) dst[OC * tx + c] = o[i][c] * inv;
    }
  }
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeTiled)f;
  }();
  return fn;
}

// rows of 16-bit values in boxes of 128 rows x 64 columns, 128-byte swizzle; rows past the end read 0
bool row_map(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, long ld) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <auto KERN, typename... A>
int launch_items(long items, int threads, int smem, cudaStream_t s, LaunchOpt o, const A &...args) {
  if (items > 0x7fffffffL) return DREAMER_ERR_UNSUPPORTED;
  return launch<KERN>(dim3((unsigned)items), dim3(threads), smem, 1, s, o, args...);
}

// the most row tiles that n_tokens rows in n_seq prompts can make, or items that find_item tells apart
long most_tiles(long n_tokens, long n_seq, long rows) {
  if (n_seq > MANY) return n_tokens / rows + n_seq;
  const long full = n_seq < n_tokens ? n_seq : n_tokens;  // prompts with a row
  return (n_tokens + full * (rows - 1)) / rows;
}

template <int D, typename... A>
int launch_tc(const PackedAttn &p, cudaStream_t s, LaunchOpt o, const A &...args) {
  using C = PkCfg<D>;
  return launch_items<packed_tc_kernel<D>>(most_tiles(p.n_tokens, p.n_seq, 128 * C::TILES) * p.Hq, C::THREADS, C::SMEM, s, o,
                                           args...);
}

// Four groups a CTA where there are at most two and a half items an SM and the prompts are longer than
// two groups' blocks on average (head dim 64; four against two groups): a prompt of 2000 tokens, 4 heads
// (252 items) 71 us against 99; four of up to 1000, 4 heads 47 against 59; the same with 16 heads (1100
// items) 175 against 144; four of up to 128, 16 heads 13 against 11.  At head dim 128 both measured
// the same.
bool long_chains(const PackedAttn &p, long items) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  return 2 * items <= 5L * sms && p.n_tokens > 128L * p.n_seq;
}

template <int D>
int launch_f32(const PackedAttn &p, cudaStream_t s, LaunchOpt o, const PackedArgs &a) {
  const long items = most_tiles(p.n_tokens, p.n_seq, 32) * p.Hq;
  if constexpr (D <= 64)
    if (long_chains(p, items))
      return launch_items<packed_f32_kernel<D, 4>>(items, F32Cfg<D, 4>::THREADS, F32Cfg<D, 4>::SMEM, s, o, a);
  return launch_items<packed_f32_kernel<D, 2>>(items, F32Cfg<D, 2>::THREADS, F32Cfg<D, 2>::SMEM, s, o, a);
}

}  // namespace

int attn_packed(const PackedAttn &p, cudaStream_t s, LaunchOpt o) {
  PackedArgs a{};
  a.cu = p.cu; a.n_seq = p.n_seq; a.n_tokens = p.n_tokens; a.Hq = p.Hq; a.G = p.Hq / p.Hkv;
  a.q = p.q; a.k = p.k; a.v = p.v; a.ldq = p.ldq; a.ldk = p.ldk; a.ldv = p.ldv;
  a.out = p.out; a.ldo = p.ldo; a.out_rows = p.out_rows;
  a.scale_log2 = p.scale * LOG2_E;
  a.err = p.err;
#ifdef DREAMER_TEST_HOOKS
  a.withhold = take_withhold();
#endif
  if (p.n_tokens == 0 || p.n_seq == 0) return DREAMER_OK;
  if (p.dtype == 1) {
    CUtensorMap tq, tk, tv;
    if (!row_map(&tq, p.q, (uint64_t)p.Hq * p.d, p.n_tokens, p.ldq) ||
        !row_map(&tk, p.k, (uint64_t)p.Hkv * p.d, p.n_tokens, p.ldk) ||
        !row_map(&tv, p.v, (uint64_t)p.Hkv * p.d, p.n_tokens, p.ldv))
      return DREAMER_ERR_CUDA;
    if (p.d == 64) return launch_tc<64>(p, s, o, tq, tk, tv, a);
    return launch_tc<128>(p, s, o, tq, tk, tv, a);
  }
  switch (p.d) {
    case 16: return launch_f32<16>(p, s, o, a);
    case 32: return launch_f32<32>(p, s, o, a);
    case 64: return launch_f32<64>(p, s, o, a);
    default: return launch_f32<128>(p, s, o, a);
  }
}

}  // namespace ops
}  // namespace dreamer

using namespace dreamer;

extern "C" int dreamer_attn_packed(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                   int64_t ldv, void *out, int64_t ldo, const int32_t *cu_seqlens, int n_seq,
                                   int n_tokens, int n_heads, int n_kv_heads, int head_dim, int dtype,
                                   float scale, int32_t *status, dreamer_stream stream) {
  if (!q || !k || !v || !out || !cu_seqlens || n_seq < 0 || n_tokens < 0) return DREAMER_ERR_ARG;
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 1) return DREAMER_ERR_ARG;
  if ((dtype != 0 && dtype != 1) || !(scale > 0.f) || !ops::scale_ok(scale)) return DREAMER_ERR_ARG;
  if (head_dim != 64 && head_dim != 128 && (dtype == 1 || (head_dim != 16 && head_dim != 32)))
    return DREAMER_ERR_UNSUPPORTED;
  const int es = dtype == 0 ? 4 : 2;
  const void *ptr[4] = {q, k, v, out};
  const int64_t ld[4] = {ldq, ldk, ldv, ldo};
  for (int i = 0; i < 4; i++) {
    const int64_t w = (int64_t)(i == 0 || i == 3 ? n_heads : n_kv_heads) * head_dim;
    if (((uintptr_t)ptr[i] & 15) || ld[i] < w || (ld[i] * es) % 16 || ld[i] * es >= (1LL << 40)) return DREAMER_ERR_ARG;
  }
  ops::PackedAttn p{q, ldq, k, ldk, v, ldv, out, ldo, cu_seqlens, n_seq, n_tokens, n_heads, n_kv_heads,
                    head_dim, dtype, scale, nullptr, status};
  return ops::attn_packed(p, (cudaStream_t)stream, ops::user_launch((cudaStream_t)stream));
}
