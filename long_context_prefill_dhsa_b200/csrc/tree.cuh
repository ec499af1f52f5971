// Shared by the kernels of the drafted-token attention (tree_attn.cu,
// tree_weight.cu): parameters, the split of the key tiles over the CTAs, the
// visibility of drafted tokens.
#pragma once
#include "cache.cuh"
#include "sm100_ptx.cuh"

namespace dhsa {

struct TreeParams {
  const __nv_bfloat16* Q;
  const int32_t *lengths, *parents, *n_draft;
  __nv_bfloat16* O;
  float* lse;
  float2* row_stat;         // per row: largest raw score and 1 / denominator, for the weight pass (null without)
  float* scores;            // [B * Hkv][rows][score_cap] raw scores for the weight pass, or null
  float* part_o;            // [piece][query tile][row_cap][128]
  float2* part_ml;          // [piece][query tile][row_cap]: reference score and sum
  const float* weight;
  float* weight_out;
  int B, Hq, Hkv, G, T, cap;
  int rows;                 // G * T
  int blocks;               // query blocks of a kv head that walk the keys
  int row_cap;              // rows of a query tile's partial
  int score_cap;            // cap rounded up to whole key tiles
  int tile;                 // slots of a key tile
  int grid;                 // CTAs that share the key tiles
  bool whole;               // items are not split: the line counts items instead of key tiles
  bool keep_k;              // K is read again after this kernel
  bool every;               // sequences without drafted tokens are walked too
  float scale, scale_log2;
  unsigned int* status;
};

namespace {

using namespace ptx;

constexpr int kMaxDrafts = 64;   // one bit of a 64-bit word each
constexpr int kMaxGroup = 64;    // query heads of one kv head
constexpr int kMaxScoreRows = 32;   // rows of a head up to which the attention keeps its scores for the weight pass
constexpr int kMaxGrid = 160;    // CTAs (one per SM) the workspace is sized for

constexpr uint32_t kTmemCols = 512;

// key tiles of each item of a sequence, and the item's length on the line
__device__ __forceinline__ int key_tiles(const TreeParams& p, const SeqLen& s) {
  return s.draft > 0 || p.every ? (s.len + s.draft + p.tile - 1) / p.tile : 0;
}
__device__ __forceinline__ int line_len(const TreeParams& p, const SeqLen& s) {
  const int n = key_tiles(p, s);
  return p.whole ? min(n, 1) : n;
}
__device__ __forceinline__ int line_len(const TreeParams& p, int b) {
  return line_len(p, seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap));
}

// The line of key tiles: sequence b's items start at `base`.
struct Line {
  long long total, start, end, base;
  int b;
};

// by one warp: the whole line's length, and the share of CTA c with the
// sequence it starts in
__device__ __forceinline__ Line find_share(const TreeParams& p, int c, int lane) {
  Line L;
  const long long per = (long long)p.Hkv * p.blocks;
  int sum = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) sum += b0 + lane < p.B ? line_len(p, b0 + lane) : 0;
  L.total = per * __reduce_add_sync(0xffffffffu, sum);
  L.start = L.total * c / p.grid;
  L.end = L.total * (c + 1) / p.grid;
  L.base = 0;
  L.b = 0;
  long long run = 0;
  for (int b0 = 0; b0 < p.B && run <= L.start; b0 += 32) {
    const int n = b0 + lane < p.B ? line_len(p, b0 + lane) : 0;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const long long from = run + (inc - n) * per, to = run + inc * per;
    const uint32_t hit = __ballot_sync(0xffffffffu, from <= L.start && L.start < to);
    if (hit) {
      const int src = __ffs(hit) - 1;
      L.b = b0 + src;
      L.base = __shfl_sync(0xffffffffu, from, src);
    }
    run += __shfl_sync(0xffffffffu, inc, 31) * per;
  }
  return L;
}

struct Piece {
  int b, h, block;
  int t0, n;            // key tiles t0 .. t0 + n - 1 of the item
  bool complete;        // they are all of its tiles
  int len, draft;
  int item;
};

// walks a CTA's share; every role does so on its own
struct Pieces {
  long long pos, end, base;
  int b;
  __device__ __forceinline__ bool next(const TreeParams& p, Piece* o) {
    if (pos >= end) return false;
    const long long per = (long long)p.Hkv * p.blocks;
    SeqLen s;
    int nt;
    for (;; ++b) {      // pos < end: a sequence with tiles follows
      s = seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap);
      nt = line_len(p, s);
      if (pos < base + nt * per) break;
      base += nt * per;
    }
    const unsigned rel = (unsigned)(pos - base);    // below 2^31 tiles of one sequence
    const unsigned in_b = rel / (unsigned)nt;
    o->b = b;
    o->h = in_b / p.blocks;
    o->block = in_b % p.blocks;
    o->t0 = rel % (unsigned)nt;
    const long long left = end - pos;
    const int n = (int)min((long long)(nt - o->t0), left);
    o->complete = n == nt;
    o->n = p.whole ? key_tiles(p, s) : n;
    o->len = s.len;
    o->draft = s.draft;
    o->item = (b * p.Hkv + o->h) * p.blocks + o->block;
    pos += n;
    return true;
  }
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// pairs of fp32 in one 64-bit register, for the packed f32x2 operations
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The drafted tokens each token sees, one bit each, by pointer doubling over
// the parents: lane l holds tokens l and l + 32.
struct Sees {
  uint64_t m0, m1;
  __device__ __forceinline__ uint64_t of(int t) const {   // all lanes, t in 0 .. 63
    const uint64_t a = __shfl_sync(0xffffffffu, m0, t & 31), c = __shfl_sync(0xffffffffu, m1, t & 31);
    return t < 32 ? a : c;
  }
};
__device__ __forceinline__ Sees tree_sees(const TreeParams& p, int b, int draft, int lane) {
  Sees s;
  const int t0 = lane, t1 = lane + 32;
  if (!p.parents) {
    s.m0 = t0 < draft ? (2ull << t0) - 1 : 0;
    s.m1 = t1 < draft ? (t1 == 63 ? ~0ull : (2ull << t1) - 1) : 0;
    return s;
  }
  int p0 = t0 < draft ? p.parents[b * p.T + t0] : -1, p1 = t1 < draft ? p.parents[b * p.T + t1] : -1;
  if (p0 < -1 || p0 >= t0 || p1 < -1 || p1 >= t1) {
    // a token without a usable parent hangs on the context
    if (p0 < -1 || p0 >= t0) p0 = -1;
    if (p1 < -1 || p1 >= t1) p1 = -1;
    raise_device_flag(p.status, DHSA_DEVFLAG_BAD_TREE);
  }
  s.m0 = t0 < draft ? 1ull << t0 : 0;
  s.m1 = t1 < draft ? 1ull << t1 : 0;
  while (__any_sync(0xffffffffu, p0 >= 0 || p1 >= 0)) {   // at most six rounds
    const Sees old = s;
    const int q0 = p0, q1 = p1;
    auto up = [&](int at) {
      const int a = __shfl_sync(0xffffffffu, q0, at & 31), c = __shfl_sync(0xffffffffu, q1, at & 31);
      return at < 32 ? a : c;
    };
    const int a0 = max(q0, 0), a1 = max(q1, 0);
    const uint64_t v0 = old.of(a0), v1 = old.of(a1);
    const int u0 = up(a0), u1 = up(a1);
    if (q0 >= 0) {
      s.m0 |= v0;
      p0 = u0;
    }
    if (q1 >= 0) {
      s.m1 |= v1;
      p1 = u1;
    }
  }
  return s;
}

struct Waits {
  volatile int* abort;
  unsigned int* status;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_test_wait(bar, parity)) return true;
    if (*abort) return false;
    if (mbar_wait_slow(bar, parity, kWaitLimitNs)) return true;
    if (mbar_test_wait(bar, parity)) return true;
    *abort = 1;
    raise_device_flag(status, DHSA_DEVFLAG_WAIT_TIMEOUT);
    return false;
  }
};

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

}  // namespace
}  // namespace dhsa
