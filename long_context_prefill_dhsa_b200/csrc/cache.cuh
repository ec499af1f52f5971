// Shared by the calls on a key/value cache (rotary.cu, tree_attn.cu, evict.cu):
// row strides, and the clamped view of a sequence's lengths.
#pragma once
#include <atomic>

#include "common.cuh"
#include "tmap.cuh"

namespace dhsa {

// strides in elements of a [B, H, rows, 128] tensor with contiguous rows
struct RowStrides {
  long long b, h, r;
};

inline RowStrides dense_strides(int H, int rows) {
  return RowStrides{(long long)H * rows * kHeadDim, (long long)rows * kHeadDim, kHeadDim};
}

// s: three host int64 or null (dense). False if a stride cannot be used: not
// a multiple of 8 elements, negative, or (distinct_rows) shorter than a row
// along a dimension with more than one entry.
inline bool read_strides(const int64_t* s, int B, int H, int rows, bool distinct_rows, RowStrides* out) {
  *out = dense_strides(H, rows);
  if (!s) return true;
  const int n[3] = {B, H, rows};
  long long* o[3] = {&out->b, &out->h, &out->r};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;   // never multiplied by anything but 0
    if (s[i] < 0 || s[i] % 8 != 0 || (distinct_rows && s[i] < kHeadDim)) return false;
    *o[i] = s[i];
  }
  return true;
}

// TMA map of a cache: boxes of 64 columns x box_rows slots of one head,
// 128-byte swizzle; slots past the capacity read as zeros.
inline bool make_cache_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, const RowStrides& s, int B, int Hkv,
                           int cap, int box_rows) {
  const cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)cap, (cuuint64_t)Hkv, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)s.r * 2, (cuuint64_t)s.h * 2, (cuuint64_t)s.b * 2};
  const cuuint32_t box[4] = {64u, (cuuint32_t)box_rows, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What is looked up or set once per device is kept in atomics: host threads
// may make their first calls at the same time, and then find the same values.

// The current device's number and SM count, looked up once per device.
inline cudaError_t this_device(int* dev, int* sms) {
  constexpr int kMost = 64;
  static std::atomic<int> count[kMost];
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= kMost) return cudaErrorInvalidDevice;
  int n = count[*dev];
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev);
    if (e != cudaSuccess) return e;
    count[*dev] = n;
  }
  *sms = n;
  return cudaSuccess;
}

// Raises a kernel's dynamic shared memory limit, once per device and kernel
// (`done`: a static array of 64 flags beside the launch).
template <typename F>
inline cudaError_t allow_smem(F* kernel, int bytes, int dev, std::atomic<bool>* done) {
  if (done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

// A sequence's cached slots and drafted tokens, clamped into the cache.
struct SeqLen {
  int len, draft;
  bool bad;
};
__device__ __forceinline__ SeqLen seq_len(const int32_t* lengths, const int32_t* n_draft, int no_draft, int b,
                                          int max_draft, int cap) {
  const int l = lengths[b], d = n_draft ? n_draft[b] : no_draft;
  SeqLen s;
  s.len = min(max(l, 0), cap);
  s.draft = min(min(max(d, 0), max_draft), cap - s.len);
  s.bad = s.len != l || s.draft != d;
  return s;
}

// Launches a kernel that may start while the one before it on the stream
// ends; the kernel itself waits (wait_for_predecessors) before it reads results.
template <typename... P, typename... A>
inline int launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

}  // namespace dhsa
