// Launchers of the handle-free attention operators, shared by their C entry points and by the
// handle's paths (dreamer.cu).  Arguments are checked by the callers; a launcher returns a
// DREAMER_* code for what only it can see (a tensor map, a CUDA error).
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/dreamer.h"

namespace dreamer {
namespace ops {

#ifdef DREAMER_TEST_HOOKS
// One copy into shared memory that the next attention kernel announces and never makes, so that the
// wait for it runs out: copy number `copy` of a warp of a CTA.
struct Withhold {
  int cta, warp, copy;
  __device__ int copy_of(unsigned c, int w) const { return (int)c == cta && w == warp ? copy : -1; }
};
inline Withhold withheld{-1, -1, -1};
inline Withhold take_withhold() {
  const Withhold w = withheld;
  withheld = Withhold{-1, -1, -1};
  return w;
}
#endif

// Launch options: programmatic dependent launch (the kernel waits by itself for what ran before on
// the stream, so its blocks may be placed meanwhile).
struct LaunchOpt {
  bool pdl = false;   // the call's first kernel
  bool next = true;   // its further ones, which follow a kernel of the call
};
// of a call on a user's stream: programmatic unless the stream is being captured, where the edge from
// an operation that is no kernel could not be
inline LaunchOpt user_launch(cudaStream_t s) {
  cudaStreamCaptureStatus st;
  LaunchOpt o;
  if (cudaStreamIsCapturing(s, &st) == cudaSuccess) o.pdl = st == cudaStreamCaptureStatusNone;
  else cudaGetLastError();
  return o;
}

// softmax in powers of two; a scale that this takes out of float32 is refused
constexpr float LOG2_E = 1.4426950408889634f;
inline bool scale_ok(float scale) { return isfinite(scale * LOG2_E); }

// Launch of one kernel (a template argument, so that what is noted of it is its own).  Its limit of
// dynamic shared memory is raised once a device, noted in bit d of `raised`, and again where a launch
// is refused all the same (a context that was reset has lost it).
template <auto KERN, typename... A>
int launch(dim3 grid, dim3 block, int smem, int cluster, cudaStream_t s, LaunchOpt o, const A &...args) {
  static std::atomic<unsigned long long> raised{0};
  const bool large = smem > 48 * 1024;
  for (bool again = false;; again = true) {
    if (large) {
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess) return DREAMER_ERR_CUDA;
      const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
      if (again || !(raised.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
          cudaGetLastError();
          return DREAMER_ERR_CUDA;
        }
        raised.fetch_or(bit, std::memory_order_release);
      }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, KERN, args...);
    if (e == cudaSuccess) return DREAMER_OK;
    cudaGetLastError();
    if (again || !large || e != cudaErrorInvalidValue) return DREAMER_ERR_CUDA;
  }
}

// ---- causal attention over packed prompts -------------------------------------------------
struct PackedAttn {
  const void *q;
  long ldq;  // row strides in elements; head j at column j * d
  const void *k;
  long ldk;
  const void *v;
  long ldv;
  void *out;
  long ldo;
  const int *cu;  // [n_seq + 1] rows of prompt i: cu[i] .. cu[i + 1] - 1
  int n_seq, n_tokens;
  int Hq, Hkv, d;
  int dtype;  // 0 float32, 1 bfloat16
  float scale;
  const int *out_rows;  // output row of token t, or null: t
  int *err;             // device error flag or null
};
int attn_packed(const PackedAttn &p, cudaStream_t s, LaunchOpt o = LaunchOpt());

// ---- 4-bit cache: one depth of one handle, or a caller's cache --------------------------
constexpr int KV4_BLOCK = 64;  // tokens of a block
constexpr int KV4_GROUP = 64;  // channels that share a (scale, offset) pair

struct Kv4Cache {
  uint8_t *data;  // [B][Hkv][cap / 64][ng * 4608]
  int B, Hkv, d, cap;
};
// bytes of one block: K codes, V codes [ng][64][32], K pairs, V pairs [ng][64][2] bf16
constexpr int kv4_block_bytes(int d) { return (d / KV4_GROUP) * KV4_BLOCK * 2 * (32 + 4); }

struct Kv4Rows {
  const void *k, *v;  // store: source rows; load: destination rows (not const there)
  long ldk, ldv;      // row strides in elements; head j at column j * d
  const int *cu;      // [B + 1] rows of sequence b: cu[b] .. cu[b + 1] - 1; null: row b is sequence b's
  const int *start;   // [B] position of a sequence's first row
  int n_rows;
  int dtype;          // 0 float32, 1 bfloat16
  int zero_rest;      // load: rows of no sequence become zeros
  int *err;           // device error flag or null
  int limit;          // positions from here on are refused (0: from the capacity on)
};
int kv4_store(const Kv4Cache &c, const Kv4Rows &r, cudaStream_t s, LaunchOpt o = LaunchOpt());
int kv4_load(const Kv4Cache &c, const Kv4Rows &r, cudaStream_t s, LaunchOpt o = LaunchOpt());

struct Kv4Attn {
  const void *q;
  long ldq;        // row stride of q in elements
  void *out;
  long ldo;
  const int *lens;  // [B]
  int len_add;      // keys of sequence b: lens[b] + len_add
  int Hq;
  int dtype;
  float scale;
  void *workspace;  // kv4_attn_workspace bytes
  int *err;
  int limit;        // more keys than this are refused (0: than the capacity)
};
// bytes of the workspace (0: none needed); any_capacity: whatever c.cap is
long kv4_attn_workspace(const Kv4Cache &c, int Hq, bool any_capacity = false);
int kv4_attn_launches(const Kv4Cache &c, int Hq, int dtype);  // kernels of a call
int kv4_attn(const Kv4Cache &c, const Kv4Attn &a, cudaStream_t s, LaunchOpt o = LaunchOpt());

}  // namespace ops
}  // namespace dreamer
