// Attention of drafted tokens over a key/value cache.
//
// Token t of sequence b sees the cached slots s < len, itself and its
// ancestors in the drafted tree; O = softmax(scale q k) v over them.
#include "cache.cuh"

namespace dhsa {
namespace {

constexpr int kMaxDrafts = 64;   // one bit of a 64-bit word each
constexpr int kMaxGroup = 64;    // query heads of one kv head

struct TreeParams {
  const __nv_bfloat16 *Q, *K, *V;
  RowStrides ks, vs;
  const int32_t *lengths, *parents, *n_draft;
  __nv_bfloat16* O;
  float *lse, *lse_ws;
  const float* weight;
  float* weight_out;
  int B, Hq, Hkv, G, T, cap;
  float scale_log2;
  unsigned int* status;
};

// drafted tokens that token t sees, one bit each
__device__ __forceinline__ uint64_t sees(const int32_t* parents, int t, unsigned int* status) {
  if (!parents) return t >= 63 ? ~0ull : (2ull << t) - 1;
  uint64_t m = 0;
  for (int a = t; a >= 0;) {
    m |= 1ull << a;
    const int up = parents[a];
    if (up < -1 || up >= a) {
      raise_device_flag(status, DHSA_DEVFLAG_BAD_TREE);
      break;
    }
    a = up;
  }
  return m;
}

__global__ void __launch_bounds__(256) tree_rows_kernel(const TreeParams p) {
  __shared__ float sm[8], sl[8], so[8][kHeadDim];
  const int t = blockIdx.x % p.T, hq = blockIdx.x / p.T % p.Hq, b = blockIdx.x / p.T / p.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqLen s = seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap);
  if (s.bad && threadIdx.x == 0) raise_device_flag(p.status, DHSA_DEVFLAG_BAD_CACHE);
  if (t >= s.draft) return;
  const uint64_t mask = sees(p.parents ? p.parents + b * p.T : nullptr, t, p.status);
  const long long row = ((long long)b * p.Hq + hq) * p.T + t;
  const int h = hq / p.G;
  const __nv_bfloat16* kb = p.K + b * p.ks.b + h * p.ks.h + lane * 4;
  const __nv_bfloat16* vb = p.V + b * p.vs.b + h * p.vs.h + lane * 4;
  float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0;
  for (int i = 0; i < 4; ++i) q[i] = __bfloat162float(p.Q[row * kHeadDim + lane * 4 + i]) * p.scale_log2;
  for (int j = warp; j < s.len + s.draft; j += 8) {
    if (j >= s.len && !((mask >> (j - s.len)) & 1)) continue;
    float d = 0;
    for (int i = 0; i < 4; ++i) d += q[i] * __bfloat162float(kb[j * p.ks.r + i]);
    for (int o2 = 16; o2 > 0; o2 >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o2);
    const float n = fmaxf(m, d), f = exp2f(m - n), e = exp2f(d - n);
    l = l * f + e;
    for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * __bfloat162float(vb[j * p.vs.r + i]);
    m = n;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int i = 0; i < 4; ++i) so[warp][lane * 4 + i] = o[i];
  __syncthreads();
  float M = -INFINITY, L = 0, x = 0;
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < 8; ++w) {
    const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M);
    L += sl[w] * f;
    if (threadIdx.x < kHeadDim) x += so[w][threadIdx.x] * f;
  }
  if (threadIdx.x < kHeadDim) p.O[row * kHeadDim + threadIdx.x] = __float2bfloat16(x / L);
  if (threadIdx.x == 0) {
    const float lse2 = M + log2f(L);
    if (p.lse) p.lse[row] = lse2 * 0.6931471805599453f;
    if (p.lse_ws) p.lse_ws[row] = lse2;
  }
}

// one warp per slot
__global__ void __launch_bounds__(256) tree_weight_kernel(const TreeParams p) {
  const long long idx = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (idx >= (long long)p.B * p.Hkv * p.cap) return;
  const int slot = (int)(idx % p.cap), h = (int)(idx / p.cap % p.Hkv), b = (int)(idx / p.cap / p.Hkv);
  const SeqLen s = seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap);
  if (slot >= s.len + s.draft) return;
  float k[4], sum = 0;
  for (int i = 0; i < 4; ++i)
    k[i] = __bfloat162float(p.K[b * p.ks.b + h * p.ks.h + slot * p.ks.r + lane * 4 + i]) * p.scale_log2;
  for (int t = 0; t < s.draft; ++t) {
    if (slot >= s.len && !((sees(p.parents ? p.parents + b * p.T : nullptr, t, p.status) >> (slot - s.len)) & 1)) continue;
    for (int g = 0; g < p.G; ++g) {
      const long long row = ((long long)b * p.Hq + h * p.G + g) * p.T + t;
      float d = 0;
      for (int i = 0; i < 4; ++i) d += k[i] * __bfloat162float(p.Q[row * kHeadDim + lane * 4 + i]);
      for (int o2 = 16; o2 > 0; o2 >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o2);
      sum += exp2f(d - p.lse_ws[row]);
    }
  }
  if (lane == 0) p.weight_out[idx] = (slot < s.len ? p.weight[idx] : 0.f) + sum;
}

}  // namespace

int tree_max_drafts() { return kMaxDrafts; }
int tree_max_group() { return kMaxGroup; }
size_t tree_ws_bytes(int B, int Hq, int Hkv, int T, int cap, bool want_weight) {
  return 256 + sizeof(float) * (size_t)B * Hq * T;
}

int launch_tree_attn(const void* Q, const void* K, const RowStrides& ks, const void* V, const RowStrides& vs, int B,
                     int Hq, int Hkv, int T, int cap, const int32_t* lengths, const int32_t* parents,
                     const int32_t* n_draft, float softmax_scale, void* O, float* lse, const float* weight,
                     float* weight_out, void* ws, unsigned int* status, cudaStream_t stream) {
  TreeParams p;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.K = static_cast<const __nv_bfloat16*>(K);
  p.V = static_cast<const __nv_bfloat16*>(V);
  p.ks = ks;
  p.vs = vs;
  p.lengths = lengths;
  p.parents = parents;
  p.n_draft = n_draft;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.lse_ws = weight_out ? static_cast<float*>(ws) : nullptr;
  p.weight = weight;
  p.weight_out = weight_out;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.T = T;
  p.cap = cap;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.status = status;
  tree_rows_kernel<<<B * Hq * T, 256, 0, stream>>>(p);
  if (weight_out)
    tree_weight_kernel<<<(unsigned)(((long long)B * Hkv * cap + 7) / 8), 256, 0, stream>>>(p);
  return launch_status();
}

}  // namespace dhsa
